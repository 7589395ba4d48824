// ts_kv_page_bounds: per page, KV head and channel, the largest and the smallest key, rounded
// outwards to the page's power-of-two grid (page_grid.cuh) and kept in bf16.
//
// The K rows of the pages are read once (block_size * d values per page and head) and 2 d bf16 are
// written, 1/8 of the bytes for 16-token bf16 pages: bound by HBM (4 x 32768 tokens, 8 KV heads, d = 128: bf16 50.9
// us, 89% of the copy rate; fp32 87, some 98%).  A warp owns one (page, head),
// whose block_size * d values are contiguous: its lanes take 16-byte chunks of consecutive rows (two
// rows of d = 128 bf16 per load instruction), keep running extremes of their channels in
// registers, and join across rows by shuffles.  No shared memory and no barrier, so a page's
// loads are all in flight at once and warps do not wait for each other.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "page_grid.cuh"

namespace ts {
namespace {

constexpr int kBoundsThreads = 256;

// Running extremes of VEC channels per lane.  The maximum and minimum instructions return the operand that is
// a number, so NaN never enters; a channel of nothing but NaN keeps (-inf, +inf) and is set to 0.  bf16 chunks
// are kept in pairs (two channels per instruction, half the shuffles).  fetch() and row() are apart so that the
// loads of several rows can be issued before the first is used.
template <typename T, int VEC>
struct Extremes {
  using Raw = typename std::conditional<VEC == 1, T, uint4>::type;
  float hi[VEC], lo[VEC];
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < VEC; ++j) hi[j] = -INFINITY, lo[j] = INFINITY;
  }
  static __device__ Raw fetch(const T* p) { return __ldg(reinterpret_cast<const Raw*>(p)); }
  __device__ void take(int j, float x) {
    hi[j] = fmaxf(hi[j], x);
    lo[j] = fminf(lo[j], x);
  }
  __device__ void row(const Raw& w) {
    if constexpr (VEC == 1) {
      take(0, static_cast<float>(w));
    } else {
      take(0, __uint_as_float(w.x));
      take(1, __uint_as_float(w.y));
      take(2, __uint_as_float(w.z));
      take(3, __uint_as_float(w.w));
    }
  }
  __device__ void from_lane(int src, bool there) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float oh = __shfl_sync(0xffffffffu, hi[j], src), ol = __shfl_sync(0xffffffffu, lo[j], src);
      if (there) {
        hi[j] = fmaxf(hi[j], oh);
        lo[j] = fminf(lo[j], ol);
      }
    }
  }
  __device__ void values(float (&h)[VEC], float (&l)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = hi[j], l[j] = lo[j];
  }
};

template <>
struct Extremes<__nv_bfloat16, 8> {
  using Raw = uint4;
  __nv_bfloat162 hi[4], lo[4];
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < 4; ++j) hi[j] = __float2bfloat162_rn(-INFINITY), lo[j] = __float2bfloat162_rn(INFINITY);
  }
  static __device__ Raw fetch(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ void row(const Raw& w) {
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = __hmax2(hi[j], x[j]);
      lo[j] = __hmin2(lo[j], x[j]);
    }
  }
  __device__ void from_lane(int src, bool there) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 oh = __shfl_sync(0xffffffffu, hi[j], src), ol = __shfl_sync(0xffffffffu, lo[j], src);
      if (there) {
        hi[j] = __hmax2(hi[j], oh);
        lo[j] = __hmin2(lo[j], ol);
      }
    }
  }
  __device__ void values(float (&h)[8], float (&l)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[2 * j] = __low2float(hi[j]), h[2 * j + 1] = __high2float(hi[j]);
      l[2 * j] = __low2float(lo[j]), l[2 * j + 1] = __high2float(lo[j]);
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
  const bool wide_out = (reinterpret_cast<uintptr_t>(bounds) & 15u) == 0;
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
  // a warp takes heads h, h + dh, ... of pages p, p + dp, ...: the items it, it + warps, ... in page-major
  // order, without a division each; the next item's page id is loaded an item ahead
  const int it0 = blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
  const int dp = warps / Hkv, dh = warps % Hkv;
  int p = p0 + it0 / Hkv, h = it0 % Hkv;
  const int end = p0 + np;
  const int32_t* row = table + static_cast<long long>(b) * max_blocks;
  int next = p < end ? __ldg(row + p) : 0;
  while (p < end) {
    const int page = next, head = h;
    p += dp;
    h += dh;
    if (h >= Hkv) {
      h -= Hkv;
      ++p;
    }
    next = __ldg(row + min(p, end - 1));
    if (page < 0 || page >= num_blocks) {
      if (lane == 0) report(status, TS_ERR_DEVICE_CHECK);
      continue;
    }
    const long long ph = static_cast<long long>(page) * Hkv + head;
    const T* base = kc + ph * bs * d;
    Extremes<T, VEC> x[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      x[j].clear();
      const int c = c0 + 32 * j;
      if (r0 < rpp && c < cpr) {
        const T* at = base + c * VEC + static_cast<long long>(r0) * d;
        const long long step = static_cast<long long>(rpp) * d;
        int r = r0;
        for (; r + 7 * rpp < bs; r += 8 * rpp, at += 8 * step) {  // eight loads in flight
          typename Extremes<T, VEC>::Raw w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) w[u] = Extremes<T, VEC>::fetch(at + u * step);
#pragma unroll
          for (int u = 0; u < 8; ++u) x[j].row(w[u]);
        }
        for (; r < bs; r += rpp, at += step) x[j].row(Extremes<T, VEC>::fetch(at));
      }
    }
    if constexpr (NJ == 1) {
      for (int o = 1; o < rpp; ++o)  // lanes of the first row gather the other rows' extremes
        x[0].from_lane((lane + o * cpr) & 31, lane + o * cpr < 32);
    }
    float amax = 0.f, xh[NJ][VEC], xl[NJ][VEC];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      x[j].values(xh[j], xl[j]);
      const bool mine = r0 == 0 && c0 + 32 * j < cpr;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const bool none = xh[j][i] < xl[j][i];
        xh[j][i] = none ? 0.f : grid_clamp(xh[j][i]);
        xl[j][i] = none ? 0.f : grid_clamp(xl[j][i]);
        if (mine) amax = fmaxf(amax, fmaxf(fabsf(xh[j][i]), fabsf(xl[j][i])));
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
        alignas(16) __nv_bfloat16 hi[VEC], lo[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          hi[i] = __float2bfloat16_rn(ceilf(xh[j][i] * up) * grid);   // exact: at most 8 bits
          lo[i] = __float2bfloat16_rn(floorf(xl[j][i] * up) * grid);
        }
        __nv_bfloat16* o = bounds + ph * 2 * d + c * VEC;
        if (VEC == 8 && wide_out) {
          *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(hi);
          *reinterpret_cast<uint4*>(o + d) = *reinterpret_cast<const uint4*>(lo);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            o[i] = hi[i];
            o[d + i] = lo[i];
          }
        }
      }
    }
  }
}

template <typename T, int VEC, int NJ>
cudaError_t go(const void* kc, int num_blocks, int bs, int Hkv, int d, const int32_t* table, int max_blocks,
               const int32_t* prefix_len, const int32_t* start_len, int B, void* bounds, int32_t* status,
               cudaStream_t stream, int num_sms) {
  // six CTAs per SM over the batch, as many as fit at once (4 x 32768 tokens: 54.5 us; five 56.3, eight, of which
  // two wait for a second round, 60.3, 64 with an item a warp 61.5)
  const long long most = (static_cast<long long>(max_blocks) * Hkv + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
  const long long want = std::max(1LL, (6LL * num_sms + B - 1) / B);
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
