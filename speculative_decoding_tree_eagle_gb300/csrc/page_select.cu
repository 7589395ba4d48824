// ts_page_select: the pages each tree node attends to, by an upper bound of its scores.
//
// For a query value q and a page's bounds lo <= k <= hi of a channel, max(q hi, q lo) is
// q+ hi + q- lo with q+ = max(q, 0), q- = min(q, 0), so the bounds of all nodes and pages are one
// matrix product per (sequence, KV head):  [q+ | q-] (m g rows, 2 d long) times [hi | lo] of every
// page.  Both sides are eight-bit whole numbers on power-of-two grids (page_grid.cuh), so bf16
// holds them and the tensor cores' fp32 sums are exact.
//
// Three launches:
//   score_kernel   tcgen05: 128 rows (whole nodes, all g heads of each) x 128 pages x 2 d per tile;
//                  the epilogue takes the maximum over the heads and writes one 32-bit key per
//                  (node, page) whose unsigned order is the score's.
//   choose_kernel  a CTA per (sequence, KV head, node): the n-th largest key by bisection over the
//                  key's bits with the keys in registers, ties by index; sets the node's bit in
//                  each kept page's word (an OR, the same in every order).
//   pack_kernel    a CTA per (sequence, KV head): the pages with any bit, ascending.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "page_grid.cuh"

namespace ts {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kRows = 128;
constexpr int kChooseThreads = 256;
constexpr int kPackThreads = 1024;
constexpr uint32_t kForced = 0xFFFFFFFFu;  // above every score's key

// Unsigned order = order of the scores (finite; -0 becomes +0).
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);
  return u ^ ((u >> 31) != 0u ? 0xFFFFFFFFu : 0x80000000u);
}

struct SelectArgs {
  const void* q;
  const __nv_bfloat16* bounds;
  const int32_t* table;
  const int32_t* prefix_len;
  uint32_t* keys;             // [B, Hkv, m, C]
  unsigned long long* dense;  // [B, Hkv, C, W]
  int32_t* pages;
  int32_t* count;
  unsigned long long* node_mask;
  int32_t* status;
  int num_blocks, bs, max_blocks, max_prefix, B, m, Hq, Hkv, g, d, C, W;
  int n, first, recent;
  int nodes_per_tile;
};

// Complete pages of the sequence, -1 for a length out of range.
__device__ __forceinline__ int complete_pages(const SelectArgs& a, int b) {
  const int L = a.prefix_len[b];
  if (L < 0 || L > a.max_prefix || L > static_cast<long long>(a.max_blocks) * a.bs) return -1;
  return L / a.bs;
}

__device__ __forceinline__ float load_q(const float* p) { return *p; }
__device__ __forceinline__ float load_q(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Shared memory of the score kernel: A and B as 128-byte-swizzled K-major chunks of 64 channels
// (first the chunks of hi / q+, then those of lo / q-), the epilogue's rows, a little state.
struct ScoreSmem {
  uint32_t off_b, off_e, off_id, off_bar, bytes;
  __host__ __device__ ScoreSmem(int chunks, int NT) {
    off_b = chunks * kRows * 128;
    off_e = off_b + chunks * NT * 128;
    off_id = off_e + 2 * kRows * 33 * 4;
    off_bar = off_id + 128 * 4;
    bytes = off_bar + 64 + 1024;
  }
};

template <typename T, int NT>
__global__ void __launch_bounds__(kScoreThreads, 1) score_kernel(const SelectArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sptr = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.z, b = bh / a.Hkv, h = bh % a.Hkv;
  const int nch = (a.d + 63) / 64;  // chunks per half
  const ScoreSmem S(2 * nch, NT);
  pdl_wait();
  const int nf = complete_pages(a, b);
  if (nf <= 0) return;
  const int n0 = blockIdx.y * a.nodes_per_tile;
  const int nodes = min(a.nodes_per_tile, a.m - n0);
  const int rows = nodes * a.g;
  if (blockIdx.y == 0) {  // the words that choose_kernel ORs into
    const long long words = static_cast<long long>(nf) * a.W;
    for (long long i = blockIdx.x * kScoreThreads + tid; i < words; i += gridDim.x * kScoreThreads)
      a.dense[static_cast<long long>(bh) * a.C * a.W + i] = 0ull;
  }
  const int ntiles = (nf + NT - 1) / NT;
  if (static_cast<int>(blockIdx.x) >= ntiles) return;

  volatile int* abort_flag = reinterpret_cast<volatile int*>(sptr + S.off_bar + 8);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sptr + S.off_bar + 16);
  const uint32_t bar = sbase + S.off_bar;
  int* s_id = reinterpret_cast<int*>(sptr + S.off_id);
  float* s_e = reinterpret_cast<float*>(sptr + S.off_e);
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_holder), NT);
    tmem_relinquish();
  }
  if (a.d % 64 != 0) {  // channels past d stay zero on both sides
    for (uint32_t i = tid * 16; i < S.off_e; i += kScoreThreads * 16)
      *reinterpret_cast<uint4*>(sptr + i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  // A: a warp per row puts the query on its grid
  for (int r = warp; r < rows; r += kScoreThreads / 32) {
    const T* qrow = static_cast<const T*>(a.q) +
                    ((static_cast<long long>(b) * a.m + n0 + r / a.g) * a.Hq + h * a.g + r % a.g) * a.d;
    float v[8], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = lane + 32 * j;
      v[j] = c < a.d ? grid_clamp(load_q(qrow + c)) : 0.f;
      amax = fmaxf(amax, fabsf(v[j]));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const int e = grid_exponent(amax);
    const float up = pow2(-e), grid = pow2(e);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = lane + 32 * j;
      if (c >= a.d) break;
      const float x = rintf(v[j] * up) * grid;  // at most eight bits: exact in bf16
      const int col = c & 63;
      unsigned char* o = sptr + (c >> 6) * (kRows * 128) + r * 128 + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2;
      *reinterpret_cast<__nv_bfloat16*>(o) = __float2bfloat16_rn(fmaxf(x, 0.f));
      *reinterpret_cast<__nv_bfloat16*>(o + nch * kRows * 128) = __float2bfloat16_rn(fminf(x, 0.f));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool vec = a.d % 8 == 0;
  bool ok = true;
  uint32_t phase = 0;
  for (int t = blockIdx.x; t < ntiles; t += gridDim.x, phase ^= 1u) {
    const int here = min(NT, nf - t * NT);
    for (int j = tid; j < here; j += kScoreThreads) {
      int id = a.table[static_cast<long long>(b) * a.max_blocks + t * NT + j];
      if (id < 0 || id >= a.num_blocks) {
        report(a.status, TS_ERR_DEVICE_CHECK);
        id = -1;
      }
      s_id[j] = id;
    }
    __syncthreads();
    if (vec) {
      const int half = a.d / 8, U = 2 * half;  // 16-byte pieces of a page's [hi | lo]
      for (int i = tid; i < here * U; i += kScoreThreads) {
        const int j = i / U, u = i - j * U, hf = u >= half ? 1 : 0, w = u - hf * half;
        const uint32_t off = S.off_b + (hf * nch + (w >> 3)) * (NT * 128) + j * 128 + (((w & 7) ^ (j & 7)) << 4);
        const int id = s_id[j];
        if (id >= 0) {
          cp_async16(sbase + off, a.bounds + (static_cast<long long>(id) * a.Hkv + h) * 2 * a.d + u * 8);
        } else {
          *reinterpret_cast<uint4*>(sptr + off) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      cp_async_wait_all();
    } else {
      for (int i = tid; i < here * 2 * a.d; i += kScoreThreads) {
        const int j = i / (2 * a.d), u = i - j * 2 * a.d, hf = u >= a.d ? 1 : 0, c = u - hf * a.d;
        const uint32_t off = S.off_b + (hf * nch + (c >> 6)) * (NT * 128) + j * 128 + ((((c & 63) >> 3) ^ (j & 7)) << 4) + (c & 7) * 2;
        const int id = s_id[j];
        *reinterpret_cast<__nv_bfloat16*>(sptr + off) =
            id >= 0 ? a.bounds[(static_cast<long long>(id) * a.Hkv + h) * 2 * a.d + u] : __float2bfloat16_rn(0.f);
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_bf16_f32(kRows, NT, 0, 0);
      for (int kk = 0; kk < 8 * nch; ++kk) {
        const uint32_t c = kk >> 2, ko = (kk & 3) * 32;
        mma_ss(tmem, sdesc_sw128(sbase + c * (kRows * 128) + ko, 16, 1024),
               sdesc_sw128(sbase + S.off_b + c * (NT * 128) + ko, 16, 1024), idesc, kk > 0 ? 1u : 0u);
      }
      tc_commit(bar);
    }
    ok = mbar_wait_warp(bar, phase, abort_flag, a.status);
    ok = __syncthreads_and(ok);
    if (!ok) break;
    tc_fence_after();
    const int q4 = warp & 3, hf = warp >> 2;
#pragma unroll 1
    for (int cg = 0; cg < NT / 32; cg += 2) {
      if (q4 * 32 < rows) {
        uint32_t u[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(q4 * 32) << 16) + 32u * (cg + hf), u);
        float* row = s_e + (hf * kRows + q4 * 32 + lane) * 33;
#pragma unroll
        for (int c = 0; c < 32; ++c) row[c] = __uint_as_float(u[c]);
      }
      __syncthreads();
      for (int i = tid; i < 64 * nodes; i += kScoreThreads) {
        const int c = i & 31, hb = (i >> 5) & 1, node = i >> 6;
        const int p = t * NT + (cg + hb) * 32 + c;
        if (p >= nf) continue;
        const float* v = s_e + (hb * kRows + node * a.g) * 33 + c;
        float best = v[0];
        for (int j = 1; j < a.g; ++j) best = fmaxf(best, v[j * 33]);
        a.keys[(static_cast<long long>(bh) * a.m + n0 + node) * a.C + p] = key_of(best);
      }
      __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 0) {
    if (!ok) {  // the products in flight land, or the limit passes, before TMEM is given back
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try(bar, phase) && global_timer_ns() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem, NT);
  }
}

// KPT keys per thread in registers; rows longer than that are read again in every round (KPT 0).
template <int KPT>
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(const SelectArgs a) {
  __shared__ int s_part[2][kChooseThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const long long row = blockIdx.x;
  const int bh = static_cast<int>(row / a.m), node = static_cast<int>(row % a.m);
  const int nf = complete_pages(a, bh / a.Hkv);
  if (nf <= 0) return;
  const uint32_t* keys = a.keys + row * a.C;
  const int head = min(a.first, nf), tail = nf - a.recent;
  auto key_at = [&](int p) -> uint32_t { return p < head || p >= tail ? kForced : __ldg(keys + p); };
  uint32_t k[KPT > 0 ? KPT : 1];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int p = tid + kChooseThreads * j;
      k[j] = p < nf ? key_at(p) : 0u;  // below every key
    }
  }
  int round = 0;
  auto at_least = [&](uint32_t x) -> int {  // pages with key >= x (x > 0), in every thread
    int c = 0;
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) c += k[j] >= x;
    } else {
      for (int p = tid; p < nf; p += kChooseThreads) c += key_at(p) >= x;
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s_part[round & 1][warp] = c;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kChooseThreads / 32; ++w) sum += s_part[round & 1][w];
    ++round;
    return sum;
  };
  unsigned long long* dense = a.dense + static_cast<long long>(bh) * a.C * a.W + (node >> 6);
  const unsigned long long bit = 1ull << (node & 63);
  auto keep = [&](int p) { atomicOr(dense + static_cast<long long>(p) * a.W, bit); };
  // the largest x with at least n keys >= x: the n-th largest key
  uint32_t x = 1u;
  int cnt = nf;
  if (nf > a.n) {
    x = 0u;
    for (int i = 31; i >= 0; --i) {
      const uint32_t y = x | (1u << i);
      const int c = at_least(y);
      if (c >= a.n) {
        x = y;
        cnt = c;
        if (c == a.n) break;
      }
    }
  }
  if (cnt <= a.n) {  // no more keys than wanted reach x
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (k[j] >= x) keep(tid + kChooseThreads * j);
    } else {
      for (int p = tid; p < nf; p += kChooseThreads)
        if (key_at(p) >= x) keep(p);
    }
    return;
  }
  // ties at x: all above it, and the first of those equal to it
  int left = a.n - at_least(x + 1u);
  for (int p0 = 0; p0 < nf; p0 += kChooseThreads) {
    const int p = p0 + tid;
    const uint32_t key = p < nf ? key_at(p) : 0u;
    if (key > x) keep(p);
    const unsigned eq = __ballot_sync(0xffffffffu, key == x && p < nf);
    if (lane == 0) s_part[round & 1][warp] = __popc(eq);
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kChooseThreads / 32; ++w) {
      before += w < warp ? s_part[round & 1][w] : 0;
      sum += s_part[round & 1][w];
    }
    ++round;
    if (((eq >> lane) & 1u) && before + __popc(eq & ((1u << lane) - 1u)) < left) keep(p);
    left -= sum;
  }
}

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const SelectArgs a) {
  __shared__ int s_warp[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int bh = blockIdx.x;
  const int nf = complete_pages(a, bh / a.Hkv);
  if (nf < 0 && tid == 0) report(a.status, TS_ERR_DEVICE_CHECK);
  const long long base = static_cast<long long>(bh) * a.C;
  int at = 0;
  for (int p0 = 0; p0 < nf; p0 += kPackThreads) {
    const int p = p0 + tid;
    unsigned long long w[4] = {0ull, 0ull, 0ull, 0ull};
    bool any = false;
    if (p < nf) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < a.W) {
          w[j] = a.dense[(base + p) * a.W + j];
          any |= w[j] != 0ull;
        }
    }
    const unsigned m = __ballot_sync(0xffffffffu, any);
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    const int c = s_warp[lane];
    int before = lane < warp ? c : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    const int sum = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (any) {
      const long long o = base + at + before + __popc(m & ((1u << lane) - 1u));
      a.pages[o] = p;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < a.W) a.node_mask[o * a.W + j] = w[j];
    }
    at += sum;
  }
  for (int p = at + tid; p < a.C; p += kPackThreads) {
    a.pages[base + p] = -1;
    for (int j = 0; j < a.W; ++j) a.node_mask[(base + p) * a.W + j] = 0ull;
  }
  if (tid == 0) a.count[bh] = at;
}

template <typename T, int NT>
cudaError_t launch_score(const SelectArgs& a, cudaStream_t stream, int num_sms) {
  const ScoreSmem S(2 * ((a.d + 63) / 64), NT);
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(score_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  });
  if (attr != cudaSuccess) return attr;
  const int groups = (a.m + a.nodes_per_tile - 1) / a.nodes_per_tile;
  const int tiles = (a.C + NT - 1) / NT;
  const long long units = static_cast<long long>(a.B) * a.Hkv * groups;
  const int gx = static_cast<int>(std::min<long long>(tiles, std::max<long long>(1, (num_sms + units - 1) / units)));
  return launch_pdl(score_kernel<T, NT>, dim3(gx, groups, a.B * a.Hkv), dim3(kScoreThreads), S.bytes, stream, a);
}

size_t keys_bytes(int B, int m, int Hkv, int C) {
  return (static_cast<size_t>(B) * Hkv * m * C * 4 + 15) / 16 * 16;
}

}  // namespace

size_t page_select_workspace_bytes(int B, int m, int Hkv, int C) {
  return keys_bytes(B, m, Hkv, C) + static_cast<size_t>(B) * Hkv * C * ((m + 63) / 64) * 8;
}

int page_select_launch(const SelectCall& c, cudaStream_t stream, int num_sms) {
  SelectArgs a;
  a.q = c.q;
  a.bounds = static_cast<const __nv_bfloat16*>(c.bounds);
  a.table = c.block_table;
  a.prefix_len = c.prefix_len;
  a.pages = c.pages;
  a.count = c.count;
  a.node_mask = reinterpret_cast<unsigned long long*>(c.node_mask);
  a.status = c.dev_status;
  a.num_blocks = c.num_blocks;
  a.bs = c.block_size;
  a.max_blocks = c.max_blocks;
  a.max_prefix = c.max_prefix;
  a.B = c.B;
  a.m = c.m;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.g = c.Hq / c.Hkv;
  a.d = c.d;
  a.C = std::max(1, c.max_prefix / c.block_size);
  a.W = (c.m + 63) / 64;
  a.n = c.n_pages;
  a.first = c.first;
  a.recent = c.recent;
  a.nodes_per_tile = kRows / a.g;
  a.keys = static_cast<uint32_t*>(c.workspace);
  a.dense = reinterpret_cast<unsigned long long*>(static_cast<char*>(c.workspace) + keys_bytes(c.B, c.m, c.Hkv, a.C));
  cudaError_t e;
  // 128 pages a tile while both operands fit shared memory, 64 for head dims above 128
  if (c.dt == TS_BF16)
    e = c.d <= 128 ? launch_score<__nv_bfloat16, 128>(a, stream, num_sms) : launch_score<__nv_bfloat16, 64>(a, stream, num_sms);
  else
    e = c.d <= 128 ? launch_score<float, 128>(a, stream, num_sms) : launch_score<float, 64>(a, stream, num_sms);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(c.B) * c.Hkv * c.m));
  if (a.C <= 8 * kChooseThreads)
    e = launch_pdl(choose_kernel<8>, grid, dim3(kChooseThreads), 0, stream, a);
  else if (a.C <= 32 * kChooseThreads)
    e = launch_pdl(choose_kernel<32>, grid, dim3(kChooseThreads), 0, stream, a);
  else
    e = launch_pdl(choose_kernel<0>, grid, dim3(kChooseThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  e = launch_pdl(pack_kernel, dim3(c.B * c.Hkv), dim3(kPackThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  return TS_OK;
}

}  // namespace ts
