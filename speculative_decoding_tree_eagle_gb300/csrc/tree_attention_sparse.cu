// ts_tree_attention_sparse, CUDA-core path: fp32 inputs (any head dim <= 256) and bf16 shapes the
// tensor-core path does not take.  fp32 arithmetic and accumulation, accurate expf.
//
// One CTA per (query head, sequence); each warp owns one node at a time and streams the keys of
// the pages that the node keeps, then the last page's prefix rows and the node's ancestors, with
// an online softmax.  Lanes split the head dimension; the dot product is a warp-shuffle sum.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace ts {
namespace {

constexpr int kSparseWarps = 4;

__device__ __forceinline__ float ld_v(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_v(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_v(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_v(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kSparseWarps * 32) sparse_simt_kernel(const SparseCall a, int W) {
  constexpr int DPL = 8;  // up to 256 / 32 head-dim elements per lane
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y;
  const int kh = h / (a.Hq / a.Hkv), bk = b * a.Hkv + kh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = a.prefix_len[b], bs = a.block_size, d = a.d, m = a.m;
  const int nu = a.count[bk];
  if (L < 0 || static_cast<long long>(L) + m > static_cast<long long>(a.max_blocks) * bs || nu < 0 || nu > a.C) {
    if (threadIdx.x == 0) report(a.dev_status, TS_ERR_DEVICE_CHECK);
    return;
  }
  const int nf = L / bs;
  const T* q = static_cast<const T*>(a.q);
  const T* kc = static_cast<const T*>(a.k_cache);
  const T* vc = static_cast<const T*>(a.v_cache);
  for (int i = warp; i < m; i += kSparseWarps) {
    const long long qo = ((static_cast<long long>(b) * m + i) * a.Hq + h) * d;
    float qv[DPL], acc[DPL];
#pragma unroll
    for (int j = 0; j < DPL; ++j) {
      const int c = lane + 32 * j;
      qv[j] = c < d ? ld_v(q + qo + c) : 0.f;
      acc[j] = 0.f;
    }
    float mloc = -INFINITY, l = 0.f;
    auto key = [&](long long row) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < DPL; ++j) {
        const int c = lane + 32 * j;
        if (c < d) s = fmaf(qv[j], ld_v(kc + row * d + c), s);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= a.scale;
      const float mnew = fmaxf(mloc, s);
      if (mnew == -INFINITY) return;
      const float corr = expf(mloc - mnew), pe = expf(s - mnew);
      l = l * corr + pe;
#pragma unroll
      for (int j = 0; j < DPL; ++j) {
        const int c = lane + 32 * j;
        if (c < d) acc[j] = acc[j] * corr + pe * ld_v(vc + row * d + c);
      }
      mloc = mnew;
    };
    auto page_row = [&](int p) -> long long {  // first K/V row of logical page p, -1 if there is none
      const int e = a.block_table[static_cast<long long>(b) * a.max_blocks + p];
      if (e < 0 || e >= a.num_blocks) {
        if (lane == 0) report(a.dev_status, TS_ERR_DEVICE_CHECK);
        return -1;
      }
      return (static_cast<long long>(e) * a.Hkv + kh) * bs;
    };
    const long long sel = static_cast<long long>(bk) * a.C;
    for (int u = 0; u < nu; ++u) {
      if (!((a.node_mask[(sel + u) * W + (i >> 6)] >> (i & 63)) & 1ull)) continue;
      const int p = a.pages[sel + u];
      if (p < 0 || p >= nf) {
        if (lane == 0) report(a.dev_status, TS_ERR_DEVICE_CHECK);
        continue;
      }
      const long long row = page_row(p);
      if (row < 0) continue;
      for (int r = 0; r < bs; ++r) key(row + r);
    }
    const uint64_t* mrow = a.mask + (static_cast<long long>(b) * m + i) * W;
    for (int pos = nf * bs; pos < L + m; ++pos) {
      if (pos >= L) {
        const int t = pos - L;
        if (!((mrow[t >> 6] >> (t & 63)) & 1ull)) continue;
      }
      const long long row = page_row(pos / bs);
      if (row >= 0) key(row + pos % bs);
    }
    const float inv = l > 0.f ? 1.f / l : l;  // no key: 0; NaN stays
#pragma unroll
    for (int j = 0; j < DPL; ++j) {
      const int c = lane + 32 * j;
      if (c < d) st_v(static_cast<T*>(a.out) + qo + c, acc[j] * inv);
    }
    if (a.lse != nullptr && lane == 0) a.lse[(static_cast<long long>(b) * m + i) * a.Hq + h] = mloc + logf(l);
  }
}

}  // namespace

int attention_sparse_simt_launch(const SparseCall& a, cudaStream_t stream) {
  const int W = (a.m + 63) / 64;
  const dim3 grid(a.Hq, a.B), block(kSparseWarps * 32);
  const cudaError_t e = a.dt == TS_F32 ? launch_pdl(sparse_simt_kernel<float>, grid, block, 0, stream, a, W)
                                       : launch_pdl(sparse_simt_kernel<__nv_bfloat16>, grid, block, 0, stream, a, W);
  count_launches(1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
