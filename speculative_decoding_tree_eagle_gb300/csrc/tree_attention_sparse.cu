// ts_tree_attention_sparse, CUDA-core path: fp32 inputs (any head dim <= 256) and bf16 shapes the
// tensor-core path does not take.  fp32 arithmetic and accumulation, accurate expf.
//
// One CTA per (node, sequence, KV head, group of up to four of its query heads): a node reads only the
// pages it keeps, and every K/V row it reads serves its group's heads.  The kept pages are listed in
// shared memory first (up to 1024 at a time), so that no warp waits for a page it will skip; then the
// eight warps take four keys at a time, lanes across the head dim.  The 4 x 4 dot products are folded
// by a reduce-scatter (16 shuffles instead of 80), so a lane ends with one (key, head) score, takes one
// exponential, and hands its weight back by a shuffle.  Each warp keeps its own running maximum, sum and
// output; they are joined through shared memory at the end.  Bound by issue slots and load latency.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace ts {
namespace {

constexpr int kWarps = 8;
constexpr int kListed = 1024;  // kept pages listed at a time
constexpr int KEYS = 4;

__device__ __forceinline__ float ld_v(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_v(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_v(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_v(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The lane that ends with item i of 4 G in the fold below: i's bits in reverse.
template <int G>
__device__ __forceinline__ constexpr int lane_of(int i) {
  int r = 0;
  for (int n = 2 * G, bit = 1; n >= 1; n /= 2, bit *= 2)
    if (i & n) r |= bit;
  return r;
}

// G query heads (1, 2 or 4) at once, DPL head-dim elements per lane.
template <typename T, int G, int DPL>
__global__ void __launch_bounds__(kWarps * 32) sparse_simt_kernel(const SparseCall a, int W) {
  __shared__ long long s_row[kListed];  // first K/V row of each listed page
  __shared__ int s_warp[kWarps];
  __shared__ float s_m[kWarps][G], s_l[kWarps][G], s_acc[kWarps][G][32 * DPL];
  pdl_wait();
  const int g = a.Hq / a.Hkv, groups = (g + G - 1) / G;
  const int node = blockIdx.x, b = blockIdx.y, kh = blockIdx.z / groups, h0 = blockIdx.z % groups * G;
  const int bk = b * a.Hkv + kh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int L = a.prefix_len[b], bs = a.block_size, d = a.d, m = a.m;
  const int nu = a.count[bk];
  if (L < 0 || static_cast<long long>(L) + m > static_cast<long long>(a.max_blocks) * bs || nu < 0 || nu > a.C) {
    if (tid == 0) report(a.dev_status, TS_ERR_DEVICE_CHECK);
    return;
  }
  const int nf = L / bs;
  const T* kc = static_cast<const T*>(a.k_cache);
  const T* vc = static_cast<const T*>(a.v_cache);
  const int32_t* table = a.block_table + static_cast<long long>(b) * a.max_blocks;
  const long long q0 = ((static_cast<long long>(b) * m + node) * a.Hq + kh * g + h0) * d;
  float q[G][DPL], acc[G][DPL], run_m[G], run_l[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    run_m[h] = -INFINITY;
    run_l[h] = 0.f;
#pragma unroll
    for (int j = 0; j < DPL; ++j) {
      const int c = lane + 32 * j;
      q[h][j] = c < d && h0 + h < g ? ld_v(static_cast<const T*>(a.q) + q0 + h * d + c) : 0.f;
      acc[h][j] = 0.f;
    }
  }
  // First row of logical page p, -1 where there is none.
  auto page_row = [&](int p) -> long long {
    const int e = table[p];
    if (e < 0 || e >= a.num_blocks) {
      report(a.dev_status, TS_ERR_DEVICE_CHECK);
      return -1;
    }
    return (static_cast<long long>(e) * a.Hkv + kh) * bs;
  };

  // Four keys (row < 0: none) into the warp's running state.  Item i = key * G + head.
  auto four = [&](const long long (&row)[KEYS]) {
    constexpr int ITEMS = KEYS * G;
    float part[ITEMS], vv[KEYS][DPL];
#pragma unroll
    for (int x = 0; x < KEYS; ++x) {
      float kk[DPL];
      const long long at = max(row[x], 0LL) * d;
#pragma unroll
      for (int j = 0; j < DPL; ++j) {
        const int c = lane + 32 * j;
        kk[j] = row[x] >= 0 && c < d ? ld_v(kc + at + c) : 0.f;
        vv[x][j] = row[x] >= 0 && c < d ? ld_v(vc + at + c) : 0.f;
      }
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < DPL; ++j) s = fmaf(q[h][j], kk[j], s);
        part[x * G + h] = s;
      }
    }
    // halve the items a lane is responsible for until one is left, then finish the sum over the other lanes
    int item = 0;
#pragma unroll
    for (int n = ITEMS / 2, bit = 1; n >= 1; n /= 2, bit *= 2) {
      const bool upper = lane & bit;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = upper ? part[i] : part[i + n], mine = upper ? part[i + n] : part[i];
        part[i] = mine + __shfl_xor_sync(0xffffffffu, send, bit);
      }
      item += upper ? n : 0;
    }
    float s = part[0];
#pragma unroll
    for (int bit = ITEMS; bit < 32; bit *= 2) s += __shfl_xor_sync(0xffffffffu, s, bit);
    // lane l now holds the score of item `item`: the bits of l in reverse, so key = the low bits of l
    const int key = item / G, head = item % G;
    long long my_row = row[0];
    float my_m = run_m[0];
#pragma unroll
    for (int x = 1; x < KEYS; ++x) my_row = key == x ? row[x] : my_row;
#pragma unroll
    for (int h = 1; h < G; ++h) my_m = head == h ? run_m[h] : my_m;
    s = my_row >= 0 ? s * a.scale : -INFINITY;
    float top = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, 1));  // over the four keys: the two lowest lane bits
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = fmaxf(top, my_m);
    const bool none = top == -INFINITY;
    const float p = none || my_row < 0 ? 0.f : expf(s - top);
    const float corr = none ? 1.f : expf(my_m - top);
    float sum = p + __shfl_xor_sync(0xffffffffu, p, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const int from = lane_of<G>(h);  // the lane with (key 0, head h)
      const float c = __shfl_sync(0xffffffffu, corr, from);
      run_m[h] = __shfl_sync(0xffffffffu, top, from);
      run_l[h] = run_l[h] * c + __shfl_sync(0xffffffffu, sum, from);
#pragma unroll
      for (int j = 0; j < DPL; ++j) acc[h][j] *= c;
#pragma unroll
      for (int x = 0; x < KEYS; ++x) {
        const float w = __shfl_sync(0xffffffffu, p, lane_of<G>(x * G + h));
        if (row[x] >= 0) {
#pragma unroll
          for (int j = 0; j < DPL; ++j) acc[h][j] = fmaf(w, vv[x][j], acc[h][j]);
        }
      }
    }
  };

  // the pages this node keeps
  const long long sel = static_cast<long long>(bk) * a.C;
  const int per_page = (bs + KEYS - 1) / KEYS;
  for (int u0 = 0; u0 < nu;) {
    // list up to kListed of them, in order: runs of 256 candidates until the list might overflow
    int listed = 0;
    while (u0 < nu && listed + kWarps * 32 <= kListed) {
      const int u = u0 + tid;
      bool keeps = u < nu && ((a.node_mask[(sel + u) * W + (node >> 6)] >> (node & 63)) & 1ull);
      long long row = -1;
      if (keeps) {
        const int p = a.pages[sel + u];
        if (p < 0 || p >= nf) report(a.dev_status, TS_ERR_DEVICE_CHECK);
        else row = page_row(p);
        keeps = row >= 0;
      }
      const unsigned mk = __ballot_sync(0xffffffffu, keeps);
      if (lane == 0) s_warp[warp] = __popc(mk);
      __syncthreads();
      int before = 0, sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? s_warp[w] : 0;
        sum += s_warp[w];
      }
      if (keeps) s_row[listed + before + __popc(mk & ((1u << lane) - 1u))] = row;
      listed += sum;
      u0 += kWarps * 32;
      __syncthreads();
    }
    for (int it = warp; it < listed * per_page; it += kWarps) {  // (at most C * bs / 4, below 2^28)
      const long long base = s_row[it / per_page];
      const int r0 = it % per_page * KEYS;
      long long row[KEYS];
#pragma unroll
      for (int x = 0; x < KEYS; ++x) row[x] = r0 + x < bs ? base + r0 + x : -1;
      four(row);
    }
    __syncthreads();  // the list is read before the next one overwrites it
  }
  // the incomplete page's prefix rows and the node's ancestors
  const uint64_t* mrow = a.mask + (static_cast<long long>(b) * m + node) * W;
  for (int pos0 = nf * bs + warp * KEYS; pos0 < L + m; pos0 += kWarps * KEYS) {
    long long row[KEYS];
    bool any = false;
#pragma unroll
    for (int x = 0; x < KEYS; ++x) {
      const int pos = pos0 + x, t = pos - L;
      const bool seen = pos < L || (pos < L + m && ((mrow[t >> 6] >> (t & 63)) & 1ull));
      const long long first = seen ? page_row(pos / bs) : -1;
      row[x] = first >= 0 ? first + pos % bs : -1;
      any |= row[x] >= 0;
    }
    if (any) four(row);
  }
  // join the warps
#pragma unroll
  for (int h = 0; h < G; ++h) {
    if (lane == 0) {
      s_m[warp][h] = run_m[h];
      s_l[warp][h] = run_l[h];
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) s_acc[warp][h][lane + 32 * j] = acc[h][j];
  }
  __syncthreads();
  for (int h = 0; h < G && h0 + h < g; ++h) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    float l = 0.f, e[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      e[w] = s_m[w][h] == -INFINITY ? (s_l[w][h] == 0.f ? 0.f : 1.f) : expf(s_m[w][h] - M);  // (a NaN sum is kept)
      l += e[w] * s_l[w][h];
    }
    const float inv = l > 0.f ? 1.f / l : l;  // no key: 0; NaN stays
    for (int c = tid; c < d; c += kWarps * 32) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (e[w] != 0.f) o += e[w] * s_acc[w][h][c];
      st_v(static_cast<T*>(a.out) + q0 + h * d + c, o * inv);
    }
    if (a.lse != nullptr && tid == 0) a.lse[(static_cast<long long>(b) * m + node) * a.Hq + kh * g + h0 + h] = M + logf(l);
  }
}

template <typename T, int G, int DPL>
cudaError_t go(const SparseCall& a, cudaStream_t stream) {
  const int groups = (a.Hq / a.Hkv + G - 1) / G;
  return launch_pdl(sparse_simt_kernel<T, G, DPL>, dim3(a.m, a.B, a.Hkv * groups), dim3(kWarps * 32), 0, stream, a, (a.m + 63) / 64);
}

template <typename T, int DPL>
cudaError_t go_heads(const SparseCall& a, cudaStream_t stream) {
  const int g = a.Hq / a.Hkv;
  return g >= 3 ? go<T, 4, DPL>(a, stream) : g == 2 ? go<T, 2, DPL>(a, stream) : go<T, 1, DPL>(a, stream);
}

template <typename T>
cudaError_t go_dim(const SparseCall& a, cudaStream_t stream) {
  return a.d <= 64 ? go_heads<T, 2>(a, stream) : a.d <= 128 ? go_heads<T, 4>(a, stream) : go_heads<T, 8>(a, stream);
}

}  // namespace

int attention_sparse_simt_launch(const SparseCall& a, cudaStream_t stream) {
  const cudaError_t e = a.dt == TS_F32 ? go_dim<float>(a, stream) : go_dim<__nv_bfloat16>(a, stream);
  count_launches(1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
