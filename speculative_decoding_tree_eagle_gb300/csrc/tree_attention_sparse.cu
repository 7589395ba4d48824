// ts_tree_attention_sparse, CUDA-core path: fp32 inputs (any head dim <= 256) and bf16 shapes the
// tensor-core path does not take.  fp32 arithmetic and accumulation, accurate expf.
//
// One CTA (or cluster) per (node, sequence, KV head, group of up to four of its query heads): a node reads only the
// pages it keeps, and every K/V row it reads serves its group's heads.  The kept pages are listed in
// shared memory first (up to 1024 at a time), so that no warp waits for a page it will skip; then the
// eight warps take four keys at a time, lanes across the head dim.  The 4 x 4 dot products are folded
// by a reduce-scatter (16 shuffles instead of 80), so a lane ends with one (key, head) score, takes one
// exponential, and hands its weight back by a shuffle.  Each warp keeps its own running maximum, sum and
// output; they are joined through shared memory at the end.  Bound by issue slots (72% of them busy, ncu), which
// nodes that keep the same page spend once each: fp32, 14 heads on 2, d = 128, 16 sequences x 32 nodes over 64 of 256
// 16-token pages take 355 us (floor 11; 365 with loads of single elements; bf16 at d = 64 248, floor 3), one node of 8
// heads on 2 15 us as a cluster of eight CTAs (39 as one; a warp per node and head that skipped pages as it met them
// took 8610 and 1119 us).
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace ts {
namespace {

constexpr int kWarps = 8;
constexpr int kListed = 1024;  // kept pages listed at a time
constexpr int KEYS = 4;

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
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

// N neighbouring elements with the widest loads (p aligned to N of them).
template <int N>
__device__ __forceinline__ void ld_n(const float* p, float (&v)[N]) {
  if constexpr (N == 2) {
    const float2 x = __ldg(reinterpret_cast<const float2*>(p));
    v[0] = x.x, v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p + i));
      v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void ld_n(const __nv_bfloat16* p, float (&v)[N]) {
  uint32_t w[N / 2];
  if constexpr (N == 2) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (N == 4) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
}

// G query heads (1, 2 or 4) at once, DPL head-dim elements per lane: neighbours, in one load (WIDE: d = 32 DPL
// and aligned tensors), or 32 apart.
template <typename T, int G, int DPL, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32) sparse_simt_kernel(const SparseCall a, int W, int cs) {
  __shared__ long long s_row[kListed];  // first K/V row of each listed page
  __shared__ int s_warp[kWarps];
  __shared__ float s_m[kWarps][G], s_l[kWarps][G], s_acc[kWarps][G][32 * DPL];
  __shared__ float s_part_m[G], s_part_l[G];  // this CTA's share (its output over s_acc[0])
  pdl_wait();
  const int g = a.Hq / a.Hkv, groups = (g + G - 1) / G;
  const int rank = blockIdx.x % cs, share = kWarps * cs;  // cs CTAs (a cluster) share a node's keys
  const int node = blockIdx.x / cs, b = blockIdx.y, kh = blockIdx.z / groups, h0 = blockIdx.z % groups * G;
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
  auto channel = [&](int j) { return WIDE ? lane * DPL + j : lane + 32 * j; };
  auto row_of = [&](const T* p, bool there, float (&v)[DPL]) {  // this lane's part of a row, zeros if there is none
    if constexpr (WIDE) {
      if (there) {
        ld_n<DPL>(p + lane * DPL, v);
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) v[j] = !WIDE && there && channel(j) < d ? ld_v(p + channel(j)) : 0.f;
  };
  float q[G][DPL], acc[G][DPL], run_m[G], run_l[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    run_m[h] = -INFINITY;
    run_l[h] = 0.f;
    row_of(static_cast<const T*>(a.q) + q0 + h * d, h0 + h < g, q[h]);
#pragma unroll
    for (int j = 0; j < DPL; ++j) acc[h][j] = 0.f;
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
      row_of(kc + at, row[x] >= 0, kk);
      row_of(vc + at, row[x] >= 0, vv[x]);
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
    // (the maxima pass over a NaN score, so one is told from no key by the score itself: it makes the sum NaN)
    const float p = s == -INFINITY ? 0.f : expf(s - top);
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
    for (int it = rank * kWarps + warp; it < listed * per_page; it += share) {  // (at most C * bs / 4, below 2^28)
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
  const long long end = static_cast<long long>(L) + m;
  for (long long pos0 = static_cast<long long>(nf) * bs + (rank * kWarps + warp) * KEYS; pos0 < end; pos0 += share * KEYS) {
    long long row[KEYS];
    bool any = false;
#pragma unroll
    for (int x = 0; x < KEYS; ++x) {
      const long long pos = pos0 + x;
      const int t = static_cast<int>(pos - L);
      const bool seen = pos < L || (pos < end && ((mrow[t >> 6] >> (t & 63)) & 1ull));
      const long long first = seen ? page_row(static_cast<int>(pos / bs)) : -1;
      row[x] = first >= 0 ? first + pos % bs : -1;
      any |= row[x] >= 0;
    }
    if (any) four(row);
  }
  // join the warps, then the CTAs of the cluster
#pragma unroll
  for (int h = 0; h < G; ++h) {
    if (lane == 0) {
      s_m[warp][h] = run_m[h];
      s_l[warp][h] = run_l[h];
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) s_acc[warp][h][channel(j)] = acc[h][j];
  }
  __syncthreads();
  // weight of a part (m, l) against the common maximum M; a NaN sum is kept, an empty part is not read
  auto weight = [](float m1, float l1, float M) { return m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : expf(m1 - M); };
#pragma unroll 1
  for (int h = 0; h < G && h0 + h < g; ++h) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    float l = 0.f, e[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      e[w] = weight(s_m[w][h], s_l[w][h], M);
      l += e[w] * s_l[w][h];
    }
    const int c = tid;  // (d <= 256 = the CTA's threads)
    float o = 0.f;
    if (c < d) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (e[w] != 0.f) o += e[w] * s_acc[w][h][c];
    }
    if (cs > 1) {
      if (c < d) s_acc[0][h][c] = o;  // (read and written by this thread only)
      if (tid == 0) {
        s_part_m[h] = M;
        s_part_l[h] = l;
      }
      continue;
    }
    const float inv = l > 0.f ? 1.f / l : l;  // no key: 0; NaN stays
    if (c < d) st_v(static_cast<T*>(a.out) + q0 + h * d + c, o * inv);
    if (a.lse != nullptr && tid == 0) a.lse[(static_cast<long long>(b) * m + node) * a.Hq + kh * g + h0 + h] = M + logf(l);
  }
  if (cs == 1) return;
  cluster_sync_all();
#pragma unroll 1
  for (int h = rank; h < G && h0 + h < g; h += cs) {  // the CTAs take the heads in turn
    float M = -INFINITY, l = 0.f, o = 0.f;
    for (int r = 0; r < cs; ++r) M = fmaxf(M, ld_dsmem_f32(dsmem_addr(smem_u32(s_part_m + h), r)));
    for (int r = 0; r < cs; ++r) {
      const float l1 = ld_dsmem_f32(dsmem_addr(smem_u32(s_part_l + h), r));
      const float e = weight(ld_dsmem_f32(dsmem_addr(smem_u32(s_part_m + h), r)), l1, M);
      l += e * l1;
      if (e != 0.f && tid < d) o += e * ld_dsmem_f32(dsmem_addr(smem_u32(&s_acc[0][h][tid]), r));
    }
    const float inv = l > 0.f ? 1.f / l : l;
    if (tid < d) st_v(static_cast<T*>(a.out) + q0 + h * d + tid, o * inv);
    if (a.lse != nullptr && tid == 0) a.lse[(static_cast<long long>(b) * m + node) * a.Hq + kh * g + h0 + h] = M + logf(l);
  }
  cluster_sync_all();  // no CTA leaves while another may still read its shared memory
}

template <typename T, int G, int DPL>
cudaError_t go(const SparseCall& a, cudaStream_t stream, int num_sms) {
  const int groups = (a.Hq / a.Hkv + G - 1) / G;
  // Few nodes: a cluster of up to eight CTAs per node, as long as they fill the GPU at most twice over (one node of 8
  // heads on 2 over 64 pages, fp32: 14.9 us against 39).
  const long long ctas = static_cast<long long>(a.m) * a.B * a.Hkv * groups;
  int cs = 1;
  while (cs < 8 && ctas * cs * 2 <= 2LL * num_sms) cs *= 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k_cache) |
                       reinterpret_cast<uintptr_t>(a.v_cache);
  const bool wide = a.d == 32 * DPL && at % 16 == 0;
  return launch_pdl_cluster(wide ? sparse_simt_kernel<T, G, DPL, true> : sparse_simt_kernel<T, G, DPL, false>,
                            dim3(a.m * cs, a.B, a.Hkv * groups), dim3(kWarps * 32), cs, stream, a, (a.m + 63) / 64, cs);
}

template <typename T, int DPL>
cudaError_t go_heads(const SparseCall& a, cudaStream_t stream, int num_sms) {
  const int g = a.Hq / a.Hkv;
  return g >= 3 ? go<T, 4, DPL>(a, stream, num_sms)
         : g == 2 ? go<T, 2, DPL>(a, stream, num_sms)
                  : go<T, 1, DPL>(a, stream, num_sms);
}

template <typename T>
cudaError_t go_dim(const SparseCall& a, cudaStream_t stream, int num_sms) {
  return a.d <= 64 ? go_heads<T, 2>(a, stream, num_sms) : a.d <= 128 ? go_heads<T, 4>(a, stream, num_sms) : go_heads<T, 8>(a, stream, num_sms);
}

}  // namespace

int attention_sparse_simt_launch(const SparseCall& a, cudaStream_t stream, int num_sms) {
  const cudaError_t e = a.dt == TS_F32 ? go_dim<float>(a, stream, num_sms) : go_dim<__nv_bfloat16>(a, stream, num_sms);
  count_launches(1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
