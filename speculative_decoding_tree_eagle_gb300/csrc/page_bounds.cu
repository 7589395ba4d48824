// ts_kv_page_bounds: per page, KV head and channel, the largest and the smallest key, rounded
// outwards to the page's power-of-two grid (page_grid.cuh) and kept in bf16.
//
// The K rows of the pages are read once (block_size * d values per page and head) and 2 d bf16 are
// written, 1/16 of the bytes for 16-token bf16 pages: bound by HBM.  A warp owns one (page, head),
// whose block_size * d values are contiguous: its lanes take 16-byte chunks of consecutive rows (two
// rows of d = 128 bf16 per load instruction), keep running extremes of their channels in
// registers, and join across rows by shuffles.  No shared memory and no barrier, so a page's
// loads are all in flight at once and warps do not wait for each other.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "page_grid.cuh"

namespace ts {
namespace {

constexpr int kBoundsThreads = 256;

// Running extremes of VEC channels per lane.  fmaxf / fminf return the operand that is a number,
// so NaN never enters; a channel of nothing but NaN keeps (-inf, +inf) and is set to 0.
template <typename T, int VEC>
struct Extremes {
  float hi[VEC], lo[VEC];
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      hi[j] = -INFINITY;
      lo[j] = INFINITY;
    }
  }
  __device__ void take(int j, float x) {
    hi[j] = fmaxf(hi[j], x);
    lo[j] = fminf(lo[j], x);
  }
  __device__ void row(const T* p) {
    if constexpr (VEC == 1) {
      take(0, static_cast<float>(*p));
    } else {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (VEC == 8) {
          take(2 * j, bf16_lo(u[j]));
          take(2 * j + 1, bf16_hi(u[j]));
        } else {
          take(j, __uint_as_float(u[j]));
        }
      }
    }
  }
};

// NJ chunks of VEC channels per lane: chunk lane % cpr (+ 32 j where a row has more than 32 chunks,
// then every lane works on the same row).
template <typename T, int VEC, int NJ>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(
    const T* __restrict__ kc, int num_blocks, int bs, int Hkv, int d, const int32_t* __restrict__ table,
    int max_blocks, const int32_t* __restrict__ prefix_len, const int32_t* __restrict__ start_len,
    __nv_bfloat16* __restrict__ bounds, int32_t* status) {
  pdl_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kBoundsThreads / 32);
  const int L = prefix_len[b], S = start_len != nullptr ? start_len[b] : 0;
  if (L < 0 || S < 0 || L > static_cast<long long>(max_blocks) * bs) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(status, TS_ERR_DEVICE_CHECK);
    return;
  }
  const int p0 = S / bs, np = L / bs - p0;
  if (np <= 0) return;
  const int cpr = d / VEC;                          // chunks per row
  const int rpp = NJ > 1 || cpr >= 32 ? 1 : 32 / cpr;  // rows per pass
  const int r0 = NJ > 1 ? 0 : lane / cpr, c0 = NJ > 1 ? lane : lane % cpr;
  const long long items = static_cast<long long>(np) * Hkv;
  for (long long it = blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const int p = p0 + static_cast<int>(it / Hkv), h = static_cast<int>(it % Hkv);
    const int page = table[static_cast<long long>(b) * max_blocks + p];
    if (page < 0 || page >= num_blocks) {
      if (lane == 0) report(status, TS_ERR_DEVICE_CHECK);
      continue;
    }
    const long long ph = static_cast<long long>(page) * Hkv + h;
    const T* base = kc + ph * bs * d;
    Extremes<T, VEC> x[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      x[j].clear();
      const int c = c0 + 32 * j;
      if (r0 < rpp && c < cpr) {
#pragma unroll 8
        for (int r = r0; r < bs; r += rpp) x[j].row(base + static_cast<long long>(r) * d + c * VEC);
      }
    }
    if constexpr (NJ == 1) {
      for (int o = 1; o < rpp; ++o) {  // lanes of the first row gather the other rows' extremes
        const int from = lane + o * cpr;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float oh = __shfl_sync(0xffffffffu, x[0].hi[j], from & 31);
          const float ol = __shfl_sync(0xffffffffu, x[0].lo[j], from & 31);
          if (from < 32) {
            x[0].hi[j] = fmaxf(x[0].hi[j], oh);
            x[0].lo[j] = fminf(x[0].lo[j], ol);
          }
        }
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int c = c0 + 32 * j;
      if (r0 == 0 && c < cpr) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const bool none = x[j].hi[i] < x[j].lo[i];
          x[j].hi[i] = none ? 0.f : grid_clamp(x[j].hi[i]);
          x[j].lo[i] = none ? 0.f : grid_clamp(x[j].lo[i]);
          amax = fmaxf(amax, fmaxf(fabsf(x[j].hi[i]), fabsf(x[j].lo[i])));
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const int e = grid_exponent(amax);
    const float up = pow2(-e), grid = pow2(e);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int c = c0 + 32 * j;
      if (r0 == 0 && c < cpr) {
        __nv_bfloat16 hi[VEC], lo[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          hi[i] = __float2bfloat16_rn(ceilf(x[j].hi[i] * up) * grid);   // exact: at most 8 bits
          lo[i] = __float2bfloat16_rn(floorf(x[j].lo[i] * up) * grid);
        }
        __nv_bfloat16* o = bounds + ph * 2 * d + c * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          o[i] = hi[i];
          o[d + i] = lo[i];
        }
      }
    }
  }
}

template <typename T, int VEC, int NJ>
cudaError_t go(const void* kc, int num_blocks, int bs, int Hkv, int d, const int32_t* table, int max_blocks,
               const int32_t* prefix_len, const int32_t* start_len, int B, void* bounds, int32_t* status,
               cudaStream_t stream, int num_sms) {
  // about eight CTAs per SM over the batch: enough loads in flight to fill HBM
  const long long most = (static_cast<long long>(max_blocks) * Hkv + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
  const long long want = std::max(1LL, (8LL * num_sms + B - 1) / B);
  return launch_pdl(page_bounds_kernel<T, VEC, NJ>, dim3(static_cast<unsigned>(std::min(most, want)), B),
                    dim3(kBoundsThreads), 0, stream, static_cast<const T*>(kc), num_blocks, bs, Hkv, d, table, max_blocks,
                    prefix_len, start_len, static_cast<__nv_bfloat16*>(bounds), status);
}

}  // namespace

int kv_page_bounds_launch(const void* k_cache, ts_dtype dt, int num_blocks, int block_size, int Hkv, int d,
                          const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                          const int32_t* start_len, int B, void* bounds, int32_t* dev_status, cudaStream_t stream,
                          int num_sms) {
  const bool al = (reinterpret_cast<uintptr_t>(k_cache) & 15u) == 0;
  cudaError_t e;
#define TS_GO(T, VEC, NJ)                                                                                        \
  go<T, VEC, NJ>(k_cache, num_blocks, block_size, Hkv, d, block_table, max_blocks, prefix_len, start_len, B, bounds, \
                 dev_status, stream, num_sms)
  // 16-byte chunks where the rows allow them (up to 32 of them in bf16, 64 in fp32), else one
  // channel at a time
  if (dt == TS_BF16) {
    e = al && d % 8 == 0 ? TS_GO(__nv_bfloat16, 8, 1) : TS_GO(__nv_bfloat16, 1, 8);
  } else {
    e = !(al && d % 4 == 0) ? TS_GO(float, 1, 8) : d <= 128 ? TS_GO(float, 4, 1) : TS_GO(float, 4, 2);
  }
#undef TS_GO
  count_launches(1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
