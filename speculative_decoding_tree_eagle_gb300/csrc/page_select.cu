// ts_page_select: the pages each tree node attends to, by an upper bound of the rounded query's scores.
//
// For a query value q and a page's bounds lo <= k <= hi of a channel, max(q hi, q lo) >= q k is
// q+ hi + q- lo with q+ = max(q, 0), q- = min(q, 0), so the bounds of all nodes and pages are one
// matrix product per (sequence, KV head):  [q+ | q-] (m g rows, 2 d long) times [hi | lo] of every
// page.  Both sides are eight-bit whole numbers on power-of-two grids (page_grid.cuh), so bf16
// holds them and the tensor cores' fp32 sums are exact.  The bounds are rounded outwards, the query to the nearest:
// the score bounds q~ k, and the query's own q k exceeds it by at most 2^(e-1) sum_c max(|hi_c|, |lo_c|), 2^e
// being the query's step (1/255 to 1/127 of its largest channel).  The rounding buys a choice that is the same in every
// order of summation; of 64 pages out of 512 it changes 0.2 to 1.1% (queries with four channels up to 300 times
// the others), and the softmax mass of the chosen pages by less than 0.0002.
//
// Three launches (one, one_node_kernel, for single nodes of few sequences):
//   score_kernel   tcgen05: 128 rows (whole nodes, all g heads of each) x 128 pages x 2 d per tile;
//                  the epilogue takes the maximum over the heads and writes one fp32 score per
//                  (node, page), NaN for pages kept anyway.
//   choose_*       a warp (or, for long rows, a CTA) per (sequence, KV head, node): the n-th largest
//                  score by bisection with the scores in registers, ties by index; sets the node's bit
//                  in each kept page's word (an OR, the same in every order).
//   pack_kernel    a CTA per (sequence, KV head): the pages with any bit, ascending.
//
// What bounds it (GB300): 4 sequences x 8 KV heads, 64 nodes of 4 heads, 2048 pages, d = 128, 128 kept
// (33.6 MB of bounds, 8.6 GFLOP): 33 us back to back.  Replayed alone from a graph, which adds some 4 us to each:
// score 19.5 us, choose 14.5 us, pack 5.5 us.  The score kernel's SMs spend half their issue slots and the tensor pipe 24%: copies, queries' rounding (5 us
// of set-up per CTA) and scores take turns on two row groups that read the same bounds.  The choosers are comparisons,
// 13 warps per SM.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "page_grid.cuh"

namespace ts {
namespace {

constexpr int kCopyThreads = 256, kKeyThreads = 512;  // score kernel: warps 0..7 and 8..23
constexpr int kIssueWarp = (kCopyThreads + kKeyThreads) / 32;
constexpr int kScoreThreads = 32 * (kIssueWarp + 1);
constexpr int kRows = 128;
constexpr int kChooseThreads = 256;      // a CTA per row
constexpr int kChooseWarpThreads = 64;   // a warp per row: small CTAs fill the SMs whatever the rows' registers
constexpr int kPackThreads = 1024;

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
  float* scores;              // [B, Hkv, m, stride], NaN for pages that do not compete
  unsigned long long* dense;  // [B, Hkv, C, W]
  int32_t* pages;
  int32_t* count;
  unsigned long long* node_mask;
  int32_t* status;
  int num_blocks, bs, max_blocks, max_prefix, B, m, Hq, Hkv, g, d, C, W;
  int n, first, recent;
  int nodes_per_tile;
  int stride;  // scores per row: C rounded up to whole tiles of 128
  int lg;      // log2 g where shuffles fold the heads, else -1
  bool q_vec;
};

// Complete pages of the sequence, -1 for a length out of range.
__device__ __forceinline__ int complete_pages(const SelectArgs& a, int b) {
  const int L = a.prefix_len[b];
  if (L < 0 || L > a.max_prefix || L > static_cast<long long>(a.max_blocks) * a.bs) return -1;
  return L / a.bs;
}

// 16 bytes to shared memory without passing registers; bytes = 0 writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

constexpr float kLeast = -3.4e38f;  // far below every score

// Pages that compete for places: those kept anyway and those past the last do not, and get NaN for a score, which
// minima, maxima and comparisons pass over (rows of scores are padded to whole tiles).
struct Compete {
  int head, n;  // pages head .. head + n - 1
  __device__ __forceinline__ float operator()(float s, int p) const {
    // (a NaN among the bounds, which ts_kv_page_bounds never writes, makes a page the last choice)
    return static_cast<unsigned>(p - head) < static_cast<unsigned>(n) ? fmaxf(s, kLeast) : __uint_as_float(0x7FFFFFFFu);
  }
};

// Scores of 32 pages out of a warp's accumulator rows, 2^LG heads per node: each step halves the columns that a
// lane is responsible for, so a node's lanes end with the maxima of 32 / 2^LG columns each.

template <int LG>
__device__ __forceinline__ void fold_out(float (&s)[32], float* scores, int stride, int r, int rows,
                                         const Compete& compete, int p) {
  constexpr int LEFT = 32 >> LG;
  const int lane = threadIdx.x & 31;
  int col = 0;
#pragma unroll
  for (int x = 0; x < LG; ++x) {
    const int H = 16 >> x;
    const bool upper = (lane >> x) & 1;
#pragma unroll
    for (int c = 0; c < H; ++c) {
      const float send = upper ? s[c] : s[c + H], mine = upper ? s[c + H] : s[c];
      s[c] = fmaxf(mine, __shfl_xor_sync(0xffffffffu, send, 1 << x));
    }
    col += upper ? H : 0;
  }
  if (r >= rows) return;
  float* o = scores + static_cast<long long>(r >> LG) * stride + p + col;
  p += col;
  if constexpr (LEFT >= 4) {
#pragma unroll
    for (int c = 0; c < LEFT; c += 4)
      *reinterpret_cast<float4*>(o + c) = make_float4(compete(s[c], p + c), compete(s[c + 1], p + c + 1),
                                                      compete(s[c + 2], p + c + 2), compete(s[c + 3], p + c + 3));
  } else {
#pragma unroll
    for (int c = 0; c < LEFT; ++c) o[c] = compete(s[c], p + c);
  }
}

// A load that stays where it is written (ahead of its use).
__device__ __forceinline__ int load_now(const int32_t* p) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One arrival per warp, after what all its lanes did (an arrival per lane would be 32 operations on one
// word, one after the other).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Head groups that are a power of two of at most 32 rows are folded by shuffles.
__host__ __device__ inline bool fold_by_shuffles(int g) { return g <= 32 && (g & (g - 1)) == 0; }

// Shared memory of the score kernel: A (the chunks of 64 channels of q+, then of q-), the B stages (a tile's
// pages by the chunks of one half, hi or lo), both 128-byte-swizzled and K-major; rows of scores for
// head groups that shuffles cannot fold; barriers.
template <int NCH, int NT>
struct ScoreCfg {
  static constexpr int ST = NCH == 4 ? 2 : 4;  // stages
  static constexpr uint32_t STAGE = NCH * NT * 128;
  static constexpr uint32_t OFF_B = 2 * NCH * kRows * 128;
  static constexpr uint32_t OFF_E = OFF_B + ST * STAGE;
  static constexpr uint32_t E_BYTES = 2 * kRows * 33 * 4;
  // full[ST] empty[ST] acc_full[2] acc_free[2] a_ready done, abort flag, TMEM address
  static constexpr uint32_t STATE = (2 * ST + 6) * 8 + 16;
  __host__ __device__ static constexpr uint32_t off_state(bool fold) { return OFF_E + (fold ? 0 : E_BYTES); }
  __host__ __device__ static constexpr uint32_t bytes(bool fold) { return off_state(fold) + STATE + 1024; }
};

// NCH chunks of 64 channels per half, NT pages per tile.  Warp roles: 0..7 copy the pages' bounds
// (cp.async, straight into the swizzled stages), 8..23 first put the queries on their grids and store
// A, then turn accumulators into keys, 24 issues the products.  Two accumulators, so a tile's products run while
// the keys of the tile before are written.
template <typename T, int NCH, int NT>
__global__ void __launch_bounds__(kScoreThreads, 1) score_kernel(const SelectArgs a) {
  using C = ScoreCfg<NCH, NT>;
  constexpr int ST = C::ST;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sptr = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.z, b = bh / a.Hkv, h = bh % a.Hkv;
  const bool fold = a.lg >= 0;
  const uint32_t state = C::off_state(fold);
  auto bar = [&](int i) -> uint32_t { return sbase + state + 8u * i; };
  auto full = [&](int s) { return bar(s); };
  auto empty = [&](int s) { return bar(ST + s); };
  auto acc_full = [&](int x) { return bar(2 * ST + x); };
  auto acc_free = [&](int x) { return bar(2 * ST + 2 + x); };
  const uint32_t a_ready = bar(2 * ST + 4), done = bar(2 * ST + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sptr + state + (2 * ST + 6) * 8);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sptr + state + (2 * ST + 6) * 8 + 8);
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), kCopyThreads);
      mbar_init(empty(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(acc_full(x), 1);
      mbar_init(acc_free(x), kKeyThreads / 32);
    }
    mbar_init(a_ready, kKeyThreads / 32);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(smem_u32(tmem_holder), 2 * NT);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  const int nf = complete_pages(a, b);
  const int n0 = blockIdx.y * a.nodes_per_tile;
  const int nodes = min(a.nodes_per_tile, a.m - n0);
  const int rows = nodes * a.g;
  const int ntiles = nf > 0 ? (nf + NT - 1) / NT : 0;
  const int t0 = blockIdx.x, step = gridDim.x;
  const int nt = t0 < ntiles ? (ntiles - t0 + step - 1) / step : 0;  // this CTA's tiles: t0, t0 + step, ...

  if (warp < kCopyThreads / 32) {
    // --------------------------------- bounds -> stages ---------------------------------
    // 8 NCH lanes take the 16-byte pieces of one page's half (zeros for channels past d and pages without an
    // id).  A thread's piece and its place in the swizzle are the same for all its pages, as these lie a
    // multiple of eight rows apart.
    constexpr int PP = 8 * NCH, STEP = kCopyThreads / PP, N = NT / STEP;
    const int piece = tid % PP, j0 = tid / PP;
    const uint32_t dst0 = sbase + C::OFF_B + (piece >> 3) * (NT * 128) + j0 * 128 + (((piece & 7) ^ (j0 & 7)) << 4);
    const bool in_d = 8 * piece < a.d, vec = a.d % 8 == 0;
    // (a piece past d copies nothing; its address is that of the first)
    const __nv_bfloat16* head = a.bounds + static_cast<long long>(h) * 2 * a.d + (in_d ? 8 * piece : 0);
    const long long page_elems = static_cast<long long>(a.Hkv) * 2 * a.d;
    const int32_t* table = a.table + static_cast<long long>(b) * a.max_blocks;
    // Physical pages: lane l of a warp holds that of the warp's page l % PW in step l / PW, loaded a tile ahead
    // (unconditionally, from a clamped place, so that nothing waits for it before its use).
    constexpr int PW = 32 / PP;
    const int my_page = warp * PW + lane % PW + STEP * (lane / PW);
    auto fetch = [&](int i) -> int { return load_now(table + min((t0 + i * step) * NT + my_page, nf - 1)); };
    int next = nt > 0 ? fetch(0) : 0;
    bool ok = true;
    for (int i = 0; i < nt && ok; ++i) {
      const bool inside = lane < PW * N && (t0 + i * step) * NT + my_page < nf;
      if (inside && (next < 0 || next >= a.num_blocks)) report(a.status, TS_ERR_DEVICE_CHECK);
      const int held = inside && next < a.num_blocks ? next : -1;
      next = fetch(i + 1);
      int id[N];
#pragma unroll
      for (int k = 0; k < N; ++k) id[k] = __shfl_sync(0xffffffffu, held, k * PW + lane / PP);
      for (int hf = 0; hf < 2; ++hf) {
        const int j = 2 * i + hf, s = j % ST;
        ok = mbar_wait_warp(empty(s), ((j / ST) & 1) ^ 1u, abort_flag, a.status);
        if (!ok) break;
        const uint32_t dst = dst0 + s * C::STAGE;
        if (vec) {
#pragma unroll
          for (int k = 0; k < N; ++k)
            cp_async16(dst + k * (STEP * 128), head + max(id[k], 0) * page_elems + hf * a.d, in_d && id[k] >= 0 ? 16 : 0);
        } else {
          // (apart from the loop above: inside it this code was skipped over in every tile, and fetching it cost
          // 6 of 25 us on the choice of 4 x 64 nodes among 2048 pages)
          for (int k = 0; k < N; ++k) {
            const int page = __shfl_sync(0xffffffffu, held, k * PW + lane / PP);
            const __nv_bfloat16* src = head + max(page, 0) * page_elems + hf * a.d;
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<__nv_bfloat16*>(sptr + (dst - sbase) + k * (STEP * 128) + 2 * e) =
                  page >= 0 && 8 * piece + e < a.d ? src[e] : __float2bfloat16_rn(0.f);
          }
        }
        // The stage's barrier counts this thread when its copies have landed.  (Signalling from here, after a wait
        // for older copies, would tie every product to the issue of later copies.)
        if (vec) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full(s)) : "memory");
        else mbar_arrive(full(s));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kIssueWarp) {
    // ------------------------------------- products -------------------------------------
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kRows, NT, 0, 0);
      const uint64_t adesc = sdesc_sw128(sbase, 16, 1024), bdesc = sdesc_sw128(sbase + C::OFF_B, 16, 1024);
      bool ok = mbar_wait(a_ready, 0, abort_flag, a.status);
      for (int i = 0; i < nt && ok; ++i) {
        if (i >= 2) ok = mbar_wait(acc_free(i & 1), ((i >> 1) & 1) ^ 1u, abort_flag, a.status);
        for (int hf = 0; hf < 2 && ok; ++hf) {
          const int j = 2 * i + hf, s = j % ST;
          ok = mbar_wait(full(s), (j / ST) & 1, abort_flag, a.status);
          if (!ok) break;
          fence_proxy_async_smem();  // the copies' writes, seen through the barrier, before the tensor cores' reads
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4 * NCH; ++kk) {  // descriptors count in 16 bytes
            const uint32_t ao = ((hf * NCH + (kk >> 2)) * (kRows * 128) + (kk & 3) * 32) >> 4;
            const uint32_t bo = (s * C::STAGE + (kk >> 2) * (NT * 128) + (kk & 3) * 32) >> 4;
            mma_ss(tmem + (i & 1) * NT, adesc + ao, bdesc + bo, idesc, (hf > 0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(empty(s));
          if (hf == 1) tc_commit(acc_full(i & 1));
        }
      }
      if (!ok) {  // the products in flight land, or the limit passes, before TMEM is given back
        tc_commit(done);
        const uint64_t start = global_timer_ns();
        while (!mbar_try(done, 0) && global_timer_ns() - start < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------- queries --------------------------------------
    const int kt = tid - kCopyThreads, kw = warp - kCopyThreads / 32;  // thread and warp among these
    if (blockIdx.y == 0) {  // the words that the choosers OR into
      const long long words = static_cast<long long>(nf) * a.W;
      for (long long i = blockIdx.x * kKeyThreads + kt; i < words; i += gridDim.x * kKeyThreads)
        a.dense[static_cast<long long>(bh) * a.C * a.W + i] = 0ull;
    }
    if (nt > 0) {
      // eight channels (a piece) per lane, LPR lanes per row.  All of a thread's pieces are first copied to where
      // its q- (and, for fp32, q+) will lie, so their latencies overlap, and then replaced one by one.
      constexpr int LPR = 8 * NCH, RPW = 32 / LPR, RSTEP = kKeyThreads / 32 * RPW;
      const int c = lane % LPR, r0 = kw * RPW + lane / LPR;
      const T* q0 = static_cast<const T*>(a.q) + ((static_cast<long long>(b) * a.m + n0) * a.Hq + h * a.g) * a.d + 8 * c;
      auto q_of = [&](int r) {
        const int node = fold ? r >> a.lg : r / a.g;
        return q0 + (static_cast<long long>(node) * (a.Hq - a.g) + r) * a.d;
      };
      auto place = [&](int r) -> uint32_t { return (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
      constexpr uint32_t NEG = NCH * kRows * 128;
      if (a.q_vec) {
        for (int r = r0; r < rows; r += RSTEP) {
          const T* q = q_of(r);
          const int bytes = 8 * c < a.d ? 16 : 0;
          const void* src = bytes != 0 ? q : a.q;
          cp_async16(sbase + place(r) + NEG, src, bytes);
          if (sizeof(T) == 4) cp_async16(sbase + place(r), static_cast<const char*>(src) + bytes, bytes);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
#pragma unroll 1
      for (int rr = kw * RPW; rr < rows; rr += RSTEP) {  // (the whole warp stays for the shuffles)
        const int r = rr + lane / LPR;
        float v[8];
        if (r >= rows) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 0.f;
        } else if (a.q_vec) {
          const uint4 w = *reinterpret_cast<const uint4*>(sptr + place(r) + NEG);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
          if (sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(u[e]), v[2 * e + 1] = bf16_hi(u[e]);
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(sptr + place(r));
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(u[e]), v[4 + e] = __uint_as_float(y[e]);
          }
        } else {
          const T* q = q_of(r);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 8 * c + e < a.d ? static_cast<float>(q[e]) : 0.f;
        }
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = grid_clamp(v[e]);
          amax = fmaxf(amax, fabsf(v[e]));
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const int e = grid_exponent(amax);
        const float up = pow2(-e), grid = pow2(e);
        uint32_t pos[4], neg[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // at most eight bits each: exact in bf16
          const float x = rintf(v[2 * i] * up) * grid, y = rintf(v[2 * i + 1] * up) * grid;
          pos[i] = pack_bf16x2(fmaxf(x, 0.f), fmaxf(y, 0.f));
          neg[i] = pack_bf16x2(fminf(x, 0.f), fminf(y, 0.f));
        }
        if (r < rows) {
          *reinterpret_cast<uint4*>(sptr + place(r)) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
          *reinterpret_cast<uint4*>(sptr + place(r) + NEG) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
        }
      }
      fence_proxy_async_smem();
      warp_arrive(a_ready);
    }
    // -------------------------------------- scores --------------------------------------
    const int q4 = kw & 3, part = kw >> 2;  // rows 32 q4 .. +31, 32 columns
    const bool mine = 32 * part < NT && q4 * 32 < rows;
    const int forced = min(a.first, max(nf, 0));
    const Compete compete{forced, max(0, nf - a.recent - forced)};
    float* scores = a.scores + (static_cast<long long>(bh) * a.m + n0) * a.stride;
    float* s_e = reinterpret_cast<float*>(sptr + C::OFF_E);
    bool ok = true;
    for (int i = 0; i < nt; ++i) {
      // (after a wait that gave up the warps still meet at the barriers below)
      if (ok) ok = mbar_wait_warp(acc_full(i & 1), (i >> 1) & 1, abort_flag, a.status);
      if (!ok && fold) break;
      tc_fence_after();
      const uint32_t acc = tmem + (i & 1) * NT + (static_cast<uint32_t>(q4 * 32) << 16);
      const int p0 = (t0 + i * step) * NT;
      float s[32];
      if (ok && mine) {
        uint32_t u[32];
        tmem_ld32(acc + 32 * part, u);
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(u[c]);
      }
      tc_fence_before();
      warp_arrive(acc_free(i & 1));  // the accumulator is in registers
      if (fold) {
        if (mine) {
          const int r = q4 * 32 + lane, p = p0 + 32 * part;
          switch (a.lg) {
            case 0: fold_out<0>(s, scores, a.stride, r, rows, compete, p); break;
            case 1: fold_out<1>(s, scores, a.stride, r, rows, compete, p); break;
            case 2: fold_out<2>(s, scores, a.stride, r, rows, compete, p); break;
            case 3: fold_out<3>(s, scores, a.stride, r, rows, compete, p); break;
            case 4: fold_out<4>(s, scores, a.stride, r, rows, compete, p); break;
            default: fold_out<5>(s, scores, a.stride, r, rows, compete, p); break;
          }
        }
      } else {
#pragma unroll 1
        for (int cg = 0; cg < NT / 64; ++cg) {  // two parts at a time go through shared memory
          if (ok && mine && (part >> 1) == cg) {
            float* row = s_e + ((part & 1) * kRows + q4 * 32 + lane) * 33;
#pragma unroll
            for (int c = 0; c < 32; ++c) row[c] = s[c];
          }
          asm volatile("bar.sync 1, %0;" ::"n"(kKeyThreads) : "memory");
          for (int x = kt; ok && x < 64 * nodes; x += kKeyThreads) {
            const int c = x & 31, hb = (x >> 5) & 1, node = x >> 6;
            const float* v = s_e + (hb * kRows + node * a.g) * 33 + c;
            float best = v[0];
            for (int y = 1; y < a.g; ++y) best = fmaxf(best, v[y * 33]);
            const int p = p0 + 32 * (2 * cg + hb) + c;
            scores[static_cast<long long>(node) * a.stride + p] = compete(best, p);
          }
          asm volatile("bar.sync 1, %0;" ::"n"(kKeyThreads) : "memory");
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * NT);
  }
}

// What a chooser needs of its row.
struct Row {
  const float* scores;
  unsigned long long* dense;  // word of this node for page 0, W apart
  unsigned long long bit;
  int nf, head, tail, need;   // pages [head, tail) compete for `need` places
};

__device__ __forceinline__ Row row_of(const SelectArgs& a, long long row) {
  Row r;
  const int bh = static_cast<int>(row / a.m), node = static_cast<int>(row % a.m);
  r.nf = complete_pages(a, bh / a.Hkv);
  r.scores = a.scores + row * a.stride;
  r.dense = a.dense + static_cast<long long>(bh) * a.C * a.W + (node >> 6);
  r.bit = 1ull << (node & 63);
  r.head = min(a.first, max(r.nf, 0));
  r.tail = max(r.nf - a.recent, r.head);
  r.need = a.n - r.head - (r.nf - r.tail);
  return r;
}

// The next bound to try between two keys: the middle of their scores for the first rounds (scores spread
// evenly halve the candidates each time), then the middle of the keys, which ends after 32 more.
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float((key >> 31) != 0u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint32_t middle(uint32_t lo, uint32_t hi, int round) {  // lo < hi; in (lo, hi]
  if (round >= 20) return lo + (hi - lo + 1u) / 2u;
  const uint32_t mid = key_of(0.5f * score_of(lo) + 0.5f * score_of(hi));
  return max(lo + 1u, min(hi, mid));
}

// n + 1 if x >= bound, else n: a comparison and a predicated addition.
__device__ __forceinline__ void count_from(float& n, float x, float bound) {
  asm("{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\t@p add.f32 %0, %0, 0f3F800000;\n\t}" : "+f"(n) : "f"(x), "f"(bound));
}
__device__ __forceinline__ float min3(float a, float b, float c) {  // (a NaN operand is ignored)
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A warp per node, the row's scores in registers (4 consecutive pages per lane and step, KPT in all):
// bisection between the smallest and the largest score until exactly `need` scores reach the bound (about
// a dozen rounds of KPT comparisons, no barrier).  The bounds tried are keys, the scores stay floats: a comparison
// and a predicated addition, two instructions on different pipes (integer keys: 17 us where this takes 14.5).  Bound
// by issue slots.  ONE (m = 1): what the node keeps is the union, so the warp writes the outputs itself.
template <int KPT, bool ONE>
__global__ void __launch_bounds__(kChooseWarpThreads) choose_warp_kernel(const SelectArgs a, long long rows) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const long long row = blockIdx.x * static_cast<long long>(kChooseWarpThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  const Row r = row_of(a, row);
  if (ONE && r.nf < 0 && lane == 0) report(a.status, TS_ERR_DEVICE_CHECK);
  if (!ONE && r.nf <= 0) return;
  auto page = [&](int j) { return (j / 4 * 32 + lane) * 4 + (j & 3); };
  const bool all = r.tail - r.head <= r.need;
  // bit j: page(j) is kept; at first all complete pages
  const int steps = max(r.nf, 0) / 128, part = max(0, min(4, r.nf - 128 * steps - 4 * lane));
  unsigned long long mine = steps >= KPT / 4 ? ~0ull >> (64 - KPT)
                                             : ((1ull << part) - 1ull) << (4 * steps) | ((1ull << (4 * steps)) - 1ull);
  if (!all) {
    const float nan = __uint_as_float(0x7FFFFFFFu);
    float k[KPT], low = nan, high = nan;
#pragma unroll
    for (int j = 0; j < KPT; j += 4) {
      const int p = page(j);
      float4 w = make_float4(nan, nan, nan, nan);
      if (p < r.nf) w = __ldg(reinterpret_cast<const float4*>(r.scores + p));
      k[j] = w.x, k[j + 1] = w.y, k[j + 2] = w.z, k[j + 3] = w.w;
    }
#pragma unroll
    for (int j = 0; j < KPT; j += 2) {
      low = min3(low, k[j], k[j + 1]);
      high = max3(high, k[j], k[j + 1]);
    }
    // (a lane may have none)
    uint32_t lo = __reduce_min_sync(0xffffffffu, isnan(low) ? 0xFFFFFFFFu : key_of(low));
    uint32_t hi = __reduce_max_sync(0xffffffffu, isnan(high) ? 0u : key_of(high));
    // invariant: at least `need` keys reach lo (cnt of them), fewer than `need` reach hi + 1 (above of them)
    int cnt = r.tail - r.head, above = 0;
    for (int round = 0; lo < hi && cnt != r.need && r.need > 0; ++round) {
      const uint32_t mid = middle(lo, hi, round);
      const float bound = score_of(mid);
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KPT; ++j) count_from(c[j & 3], k[j], bound);
      const int n = __reduce_add_sync(0xffffffffu, static_cast<int>((c[0] + c[1]) + (c[2] + c[3])));
      if (n >= r.need) {
        lo = mid;
        cnt = n;
      } else {
        hi = mid - 1u;
        above = n;
      }
    }
    // those kept without a comparison have NaN and are not below the bound either
    const float bound = r.need > 0 ? score_of(lo) : INFINITY;
    unsigned long long reach = 0ull;
#pragma unroll
    for (int j = 0; j < KPT; ++j)
      if (!(k[j] < bound)) reach |= 1ull << j;
    if (r.need > 0 && cnt != r.need) {  // ties at lo == hi: of the keys equal to it only the first
      unsigned long long eq = 0ull;
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (k[j] == bound) eq |= 1ull << j;
      reach &= ~eq;
      int left = r.need - above;
#pragma unroll 1
      for (int s = 0; s < KPT / 4 && left > 0; ++s) {
        const unsigned four = static_cast<unsigned>(eq >> (4 * s)) & 0xFu;
        int before = __popc(four);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        const int sum = __shfl_sync(0xffffffffu, before, 31);
        before -= __popc(four);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (((four >> e) & 1u) != 0u && before + __popc(four & ((1u << e) - 1u)) < left) reach |= 1ull << (4 * s + e);
        left -= sum;
      }
    }
    mine &= reach;
  }
  if constexpr (!ONE) {
    while (mine != 0ull) {
      const int j = __ffsll(static_cast<long long>(mine)) - 1;
      mine &= mine - 1ull;
      atomicOr(r.dense + static_cast<long long>(page(j)) * a.W, r.bit);
    }
  } else {
    int32_t* pages = a.pages + row * a.C;
    unsigned long long* words = a.node_mask + row * a.C;
    int at = 0;
#pragma unroll 1
    for (int s = 0; s < KPT / 4 && 128 * s < r.nf; ++s) {
      unsigned four = static_cast<unsigned>(mine >> (4 * s)) & 0xFu;
      int before = __popc(four);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      const int sum = __shfl_sync(0xffffffffu, before, 31);
      int o = at + before - __popc(four);
      for (; four != 0u; four &= four - 1u, ++o) {
        pages[o] = page(4 * s + __ffs(four) - 1);
        words[o] = 1ull;
      }
      at += sum;
    }
    for (int p = at + lane; p < a.C; p += 32) {
      pages[p] = -1;
      words[p] = 0ull;
    }
    if (lane == 0) a.count[row] = at;
  }
}

// A CTA per node for longer rows: the same bisection, KPT keys per thread in registers, or read
// again in every round (KPT 0).
template <int KPT>
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(const SelectArgs a) {
  __shared__ int s_part[2][kChooseThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const Row r = row_of(a, blockIdx.x);
  if (r.nf <= 0) return;
  auto keep = [&](int p) { atomicOr(r.dense + static_cast<long long>(p) * a.W, r.bit); };
  const bool all = r.tail - r.head <= r.need;
  for (int p = tid; p < r.nf; p += kChooseThreads)
    if (p < r.head || p >= r.tail || all) keep(p);
  if (all || r.need <= 0) return;
  uint32_t k[KPT > 0 ? KPT : 1];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int p = r.head + tid + kChooseThreads * j;
      k[j] = p < r.tail ? key_of(__ldg(r.scores + p)) : 0u;  // below every key
    }
  }
  int round = 0;
  auto sum_up = [&](int c) -> int {
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s_part[round & 1][warp] = c;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kChooseThreads / 32; ++w) sum += s_part[round & 1][w];
    ++round;
    return sum;
  };
  auto at_least = [&](uint32_t x) -> int {  // keys >= x (x > 0), in every thread
    int c = 0;
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) c += k[j] >= x;
    } else {
      for (int p = r.head + tid; p < r.tail; p += kChooseThreads) c += key_of(__ldg(r.scores + p)) >= x;
    }
    return sum_up(c);
  };
  uint32_t lo = key_of(kLeast), hi = key_of(-kLeast);
  int cnt = r.tail - r.head;
  for (int step = 0; lo < hi && cnt != r.need; ++step) {
    const uint32_t mid = middle(lo, hi, step + 20);
    const int c = at_least(mid);
    if (c >= r.need) {
      lo = mid;
      cnt = c;
    } else {
      hi = mid - 1u;
    }
  }
  // all above lo, and of those equal to it the first `left` (all of them when cnt == need)
  int left = cnt == r.need ? cnt : r.need - at_least(lo + 1u);
  for (int p0 = r.head; p0 < r.tail; p0 += kChooseThreads) {
    const int p = p0 + tid;
    const uint32_t key = p < r.tail ? key_of(__ldg(r.scores + p)) : 0u;
    if (cnt == r.need) {
      if (key >= lo) keep(p);
      continue;
    }
    if (key > lo) keep(p);
    const unsigned eq = __ballot_sync(0xffffffffu, key == lo);
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

// One node per sequence: a cluster of eight CTAs per (sequence, KV head) scores all its pages on the CUDA
// cores, each key goes straight into the shared memory of the cluster's first CTA, and that one chooses and
// writes the outputs.  One launch and nothing in the workspace.
//
// LPP lanes hold a page's channels, eight each, with the queries' values in registers, G heads (a smaller group
// repeats its last head, which changes no maximum).  Up to four heads are kept as q+ and q- (two FMA per head and
// channel); eight as q, the bound picked by its sign (three instructions), to stay within the registers.
//
// What bounds it: latency and code that runs once.  8 KV heads of 4 heads, 2048 pages, d = 128 (8.4 MB): 19000
// cycles of the first CTA, 4000 of them for the queries (each warp rounding all heads by itself: 6000), 6500 for the
// scores (64 of 152 SMs), 4000 for the bound (bisection: 7400, of 600 each round) and 2500 for the outputs.
constexpr int kOneCtas = 8, kOneThreads = 512, kOneWarps = kOneThreads / 32;
constexpr int kOnePages = 8192;                     // keys the first CTA holds
static_assert(kOnePages / kOneThreads * kOneWarps <= kOneThreads, "a count per warp and step, one per thread");
constexpr int kOneBins = kOneThreads;
constexpr int kOneAhead = 2;                        // pages whose bounds a lane has on their way

template <typename T, int LPP, int G>
__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads, 1) one_node_kernel(const SelectArgs a) {
  __shared__ uint32_t s_key[kOnePages];
  __shared__ int s_cnt[kOneThreads];
  __shared__ int s_part[2][kOneWarps];
  __shared__ float4 s_q4[G <= 4 ? 2 * G : G][2 * LPP];
  __shared__ int s_bin[kOneBins];
  __shared__ uint32_t s_near[32], s_high[2][kOneWarps];
  __shared__ int s_found[4];
  auto s_q = reinterpret_cast<float (*)[8 * LPP]>(s_q4);
  constexpr int PPW = 32 / LPP;  // pages per warp and step
  constexpr int STEP = kOneCtas * kOneWarps * PPW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank()), bh = blockIdx.x / kOneCtas, b = bh / a.Hkv, h = bh % a.Hkv;
  pdl_wait();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int32_t* table = a.table + static_cast<long long>(b) * a.max_blocks;
  const int last = min(a.C, a.max_blocks) - 1;  // the table is read ahead of the length, from a clamped place
  const int p0 = (rank * kOneWarps + warp) * PPW + lane / LPP;
  int ids[kOneAhead];
#pragma unroll
  for (int u = 0; u < kOneAhead; ++u) ids[u] = load_now(table + min(p0 + u * STEP, last));
  const int nf = complete_pages(a, b);
  const int c = lane % LPP;
  const bool in_d = 8 * c < a.d;
  const __nv_bfloat16* bounds = a.bounds + static_cast<long long>(h) * 2 * a.d + (in_d ? 8 * c : 0);
  const long long page_elems = static_cast<long long>(a.Hkv) * 2 * a.d;
  uint4 hi[kOneAhead], lo[kOneAhead];
  auto load = [&](int s0) {  // the bounds of pages s0 + p0 + u * STEP, whose ids are held; then the ids after them
#pragma unroll
    for (int u = 0; u < kOneAhead; ++u) {
      hi[u] = lo[u] = make_uint4(0u, 0u, 0u, 0u);
      if (s0 + p0 + u * STEP < nf) {
        if (ids[u] >= 0 && ids[u] < a.num_blocks) {
          const __nv_bfloat16* at = bounds + ids[u] * page_elems;
          if (in_d) {
            hi[u] = __ldg(reinterpret_cast<const uint4*>(at));
            lo[u] = __ldg(reinterpret_cast<const uint4*>(at + a.d));
          }
        } else {
          report(a.status, TS_ERR_DEVICE_CHECK);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kOneAhead; ++u) ids[u] = load_now(table + min(s0 + p0 + (kOneAhead + u) * STEP, last));
  };
  load(0);

  // Queries on their grids: a warp per head, for all warps.
  constexpr bool SPLIT = G <= 4;
  if (warp < G) {
    constexpr int E = LPP / 4;  // channels per lane
    const int d0 = lane * E;
    const T* q = static_cast<const T*>(a.q) + (static_cast<long long>(b) * a.Hq + h * a.g + min(warp, a.g - 1)) * a.d;
    float v[E], amax = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = d0 + e < a.d ? grid_clamp(static_cast<float>(q[d0 + e])) : 0.f;
      amax = fmaxf(amax, fabsf(v[e]));
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // (not negative)
    const int e2 = grid_exponent(amax);
    const float up = pow2(-e2), grid = pow2(e2);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = rintf(v[e] * up) * grid;
      s_q[warp][d0 + e] = SPLIT ? fmaxf(x, 0.f) : x;
      if constexpr (SPLIT) s_q[G + warp][d0 + e] = fminf(x, 0.f);
    }
  }
  s_bin[tid] = 0;
  if (tid < 4) s_found[tid] = 0;
  __syncthreads();
  uint64_t qp[G][4], qn[SPLIT ? G : 1][4];  // two channels each
#pragma unroll
  for (int x = 0; x < G; ++x) {
    auto fetch = [&](int row, uint64_t (&to)[4]) {
      const ulonglong2* from = reinterpret_cast<const ulonglong2*>(s_q[row] + 8 * c);
      const ulonglong2 f = from[0], g = from[1];
      to[0] = f.x, to[1] = f.y, to[2] = g.x, to[3] = g.y;
    };
    fetch(x, qp[x]);
    if constexpr (SPLIT) fetch(G + x, qn[x]);
  }

  // ------------------------------------------- keys --------------------------------------------
  const int head = min(a.first, max(nf, 0)), tail = max(nf - a.recent, head), need = a.n - head - (nf - tail);
  const bool all = tail - head <= need;
  const uint32_t to = dsmem_addr(smem_u32(s_key), 0);
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA runs: its shared memory can be written
  for (int s0 = 0; s0 < nf; s0 += kOneAhead * STEP) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int u = 0; u < kOneAhead; ++u) {
      uint64_t acc2[G];
#pragma unroll
      for (int x = 0; x < G; ++x) acc2[x] = 0ull;
      const uint32_t wh[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w}, wl[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float h0 = bf16_lo(wh[e]), h1 = bf16_hi(wh[e]), l0 = bf16_lo(wl[e]), l1 = bf16_hi(wl[e]);
#pragma unroll
        for (int x = 0; x < G; ++x) {
          if constexpr (SPLIT) {
            acc2[x] = fma_f32x2(qn[x][e], pack_f32x2(l0, l1), fma_f32x2(qp[x][e], pack_f32x2(h0, h1), acc2[x]));
          } else {
            float q0, q1;
            unpack_f32x2(qp[x][e], q0, q1);
            acc2[x] = fma_f32x2(qp[x][e], pack_f32x2(q0 >= 0.f ? h0 : l0, q1 >= 0.f ? h1 : l1), acc2[x]);
          }
        }
      }
      float acc[G];
#pragma unroll
      for (int x = 0; x < G; ++x) {
        float a0, a1;
        unpack_f32x2(acc2[x], a0, a1);
        acc[x] = a0 + a1;
      }
      // sums over the page's lanes: the first steps also divide the heads among the lanes
      int off = LPP / 2;
#pragma unroll
      for (int n = G; n > 1; n >>= 1, off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int x = 0; x < n / 2; ++x) {
          const float send = upper ? acc[x] : acc[x + n / 2], mine = upper ? acc[x + n / 2] : acc[x];
          acc[x] = mine + __shfl_xor_sync(0xffffffffu, send, off);
        }
      }
      float sum = acc[0];
#pragma unroll
      for (int o = LPP / (2 * G); o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
      for (int o = LPP / 2; o >= LPP / G; o >>= 1) sum = fmaxf(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      const int p = s0 + p0 + u * STEP;
      if (c == 0 && p < nf) asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + 4u * p), "r"(p >= head && p < tail ? key_of(fmaxf(sum, kLeast)) : 0u) : "memory");
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  int32_t* pages = a.pages + static_cast<long long>(bh) * a.C;
  unsigned long long* words = a.node_mask + static_cast<long long>(bh) * a.C;
  const int kept = nf <= 0 ? 0 : all ? nf : a.n;
  for (int p = kept + rank * kOneThreads + tid; p < a.C; p += kOneCtas * kOneThreads) {
    pages[p] = -1;
    words[p] = 0ull;
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank != 0) return;

  // ------------------------------------------ choice -------------------------------------------
  if (tid == 0) {
    a.count[bh] = kept;
    if (nf < 0) report(a.status, TS_ERR_DEVICE_CHECK);
  }
  if (nf <= 0) return;
  // (The loops from here on are not unrolled and read the keys from shared memory: this code runs once, by one CTA,
  // and what it costs is fetching it.)
  const int nk = (nf + kOneThreads - 1) / kOneThreads;  // pages tid + 512 j, j < nk
  auto key_at = [&](int j) -> uint32_t {
    const int p = tid + kOneThreads * j;
    return p < nf ? s_key[p] : 0u;
  };
  int round = 0;
  auto sum_up = [&](int v) -> int {  // of all threads, in every thread
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) s_part[round & 1][warp] = v;
    __syncthreads();
    const int t = lane < kOneWarps ? s_part[round & 1][lane] : 0;
    ++round;
    return __reduce_add_sync(0xffffffffu, t);
  };
  auto sum_before = [&](int v) -> int {  // of the threads before this one
    int at = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    if (lane == 31) s_part[round & 1][warp] = at;
    __syncthreads();
    const int t = lane < warp ? s_part[round & 1][lane % kOneWarps] : 0;
    ++round;
    return at - v + __reduce_add_sync(0xffffffffu, t);
  };
  // Positions of flagged pages (flags bit j: page tid + 512 j) among all flagged ones, in page order.
  auto count_all = [&](uint32_t flags) {
    __syncthreads();
    s_cnt[tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < nk; ++j) {
      const unsigned m = __ballot_sync(0xffffffffu, (flags >> j) & 1u);
      if (lane == 0) s_cnt[j * kOneWarps + warp] = __popc(m);
    }
    __syncthreads();
    const int at = sum_before(s_cnt[tid]);
    s_cnt[tid] = at;
    __syncthreads();
  };
  auto position = [&](int j, uint32_t flags) -> int {  // (every lane of the warp)
    const unsigned m = __ballot_sync(0xffffffffu, (flags >> j) & 1u);
    return s_cnt[j * kOneWarps + warp] + __popc(m & ((1u << lane) - 1u));
  };
  uint32_t lo_key = 1u, hi_key = 0xFFFFFFFFu, keep = 0u;
  int cnt = tail - head, above = 0;
  const bool choose = !all && need > 0;
  if (choose) {
    uint32_t low = 0xFFFFFFFFu, high = 0u;
    auto of_all = [&]() {  // smallest low and largest high
      low = __reduce_min_sync(0xffffffffu, low);
      high = __reduce_max_sync(0xffffffffu, high);
      if (lane == 0) s_part[round & 1][warp] = static_cast<int>(low), s_high[round & 1][warp] = high;
      __syncthreads();
      lo_key = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(s_part[round & 1][lane % kOneWarps]));
      hi_key = __reduce_max_sync(0xffffffffu, s_high[round & 1][lane % kOneWarps]);
      ++round;
    };
#pragma unroll 1
    for (int j = 0; j < nk; ++j) {
      const uint32_t k = key_at(j);
      low = min(low, k - 1u);  // (a key of 0 becomes the largest)
      high = max(high, k);
    }
    of_all();
    ++lo_key;
    // invariant: at least `need` keys reach lo_key (cnt of them), fewer than `need` reach hi_key + 1 (above of them)
    if (lo_key < hi_key && cnt != need) {
      // The counts of 512 equal ranges of scores find the range that holds the need-th key (rounding keeps the
      // order), and where at most 32 keys lie in it, those are compared with one another.
      const float s0 = score_of(lo_key), scale = (kOneBins - 1) / (score_of(hi_key) - s0);
      auto bin = [&](uint32_t x) { return max(0, min(kOneBins - 1, static_cast<int>((score_of(x) - s0) * scale))); };
#pragma unroll 1
      for (int j = 0; j < nk; ++j) {
        const uint32_t k = key_at(j);
        if (k != 0u) atomicAdd(s_bin + bin(k), 1);
      }
      __syncthreads();
      const int v = s_bin[kOneBins - 1 - tid];  // the highest range first
      const int at = sum_before(v);
      if (at < need && at + v >= need) s_found[0] = kOneBins - 1 - tid, s_found[1] = at, s_found[2] = v, s_found[3] = 0;
      __syncthreads();
      const int range = s_found[0], n = s_found[2];
      above = s_found[1];
      cnt = above + n;
      low = 0xFFFFFFFFu, high = 0u;
#pragma unroll 1
      for (int j = 0; j < nk; ++j) {
        const uint32_t k = key_at(j);
        if (k == 0u || bin(k) != range) continue;
        low = min(low, k);
        high = max(high, k);
        if (n <= 32) s_near[min(atomicAdd(s_found + 3, 1), 31)] = k;
      }
      __syncwarp();
      if (n <= 32) {
        __syncthreads();
        // (every warp by itself: the key that fewer than `need` keys exceed and at least `need` reach)
        const uint32_t x = lane < n ? s_near[lane] : 0u;
        int more = 0, reach = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t y = s_near[i];
          more += y > x;
          reach += y >= x;
        }
        const unsigned m = __ballot_sync(0xffffffffu, lane < n && above + more < need && above + reach >= need);
        const int who = __ffs(m) - 1;
        lo_key = hi_key = __shfl_sync(0xffffffffu, x, who);
        cnt = above + __shfl_sync(0xffffffffu, reach, who);
        above += __shfl_sync(0xffffffffu, more, who);
      } else {
        of_all();
      }
    }
#pragma unroll 1
    for (int step = 0; lo_key < hi_key && cnt != need; ++step) {
      const uint32_t mid = middle(lo_key, hi_key, step);
      int v = 0;
#pragma unroll 1
      for (int j = 0; j < nk; ++j) v += key_at(j) >= mid;
      v = sum_up(v);
      if (v >= need) {
        lo_key = mid;
        cnt = v;
      } else {
        hi_key = mid - 1u;
        above = v;
      }
    }
  }
  uint32_t equal = 0u;  // bit j: page tid + 512 j
#pragma unroll 1
  for (int j = 0; j < nk; ++j) {
    const int p = tid + kOneThreads * j;
    const uint32_t k = key_at(j);
    const bool tie = choose && cnt != need && k == lo_key;  // at lo_key == hi_key: only the first of them
    const bool in = all || p < head || p >= tail || (choose && k >= lo_key);
    if (p < nf && in && !tie) keep |= 1u << j;
    if (tie) equal |= 1u << j;
  }
  if (choose && cnt != need) {
    count_all(equal);
#pragma unroll 1
    for (int j = 0; j < nk; ++j)
      if (position(j, equal) < need - above && ((equal >> j) & 1u)) keep |= 1u << j;
  }
  count_all(keep);
#pragma unroll 1
  for (int j = 0; j < nk; ++j) {
    const int o = position(j, keep);
    if ((keep >> j) & 1u) {
      pages[o] = tid + kOneThreads * j;
      words[o] = 1ull;
    }
  }
}

template <typename T, int LPP>
cudaError_t launch_one(const SelectArgs& a, cudaStream_t stream) {
  const dim3 grid(kOneCtas * a.B * a.Hkv), block(kOneThreads);
  if (a.g == 1) return launch_pdl(one_node_kernel<T, LPP, 1>, grid, block, 0, stream, a);
  if (a.g == 2) return launch_pdl(one_node_kernel<T, LPP, 2>, grid, block, 0, stream, a);
  if (a.g <= 4) return launch_pdl(one_node_kernel<T, LPP, 4>, grid, block, 0, stream, a);
  return launch_pdl(one_node_kernel<T, LPP, 8>, grid, block, 0, stream, a);
}

template <typename T>
cudaError_t launch_one(const SelectArgs& a, cudaStream_t stream) {
  if (a.d <= 64) return launch_one<T, 8>(a, stream);
  return a.d <= 128 ? launch_one<T, 16>(a, stream) : launch_one<T, 32>(a, stream);
}

// Whether one_node_kernel takes the call: while its clusters run at once and a cluster's work is small.  Against the
// score and choice kernels, d = 128, in us on the device (from Python 20 and 25):
//   8 clusters of 4 heads: 64 pages 8.5 and 12.4, 2048 pages 12.5 and 18.6; 16 clusters: 12.4 and 12.4, 18.6 and 18.7;
//   32 clusters: 14.7 and 12.4, 24.8 and 20.7; 8 clusters of 8 heads, 2048 pages: 18.5 and 16.7;
//   one of 8 heads, 8192 pages: 48 and 27.
bool one_node(int B, int m, int Hq, int Hkv, int d, int C) {
  constexpr long long kClusters = 16, kWork = 1 << 20;  // kWork: pages x heads x channels, as the kernel rounds them up
  const int g = Hq / Hkv, heads = g <= 2 ? g : g <= 4 ? 4 : 8, channels = d <= 64 ? 64 : d <= 128 ? 128 : 256;
  return m == 1 && d % 8 == 0 && g <= 8 && C <= kOnePages && static_cast<long long>(B) * Hkv <= kClusters &&
         static_cast<long long>(C) * heads * channels <= kWork;
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

template <typename T, int NCH, int NT>
cudaError_t launch_score(const SelectArgs& a, cudaStream_t stream, int num_sms) {
  using C = ScoreCfg<NCH, NT>;
  static_assert(C::bytes(false) <= 232448, "shared memory budget");
  static std::atomic<uint64_t> done{0};
  const cudaError_t attr = once_per_device(done, [] {
    return cudaFuncSetAttribute(score_kernel<T, NCH, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::bytes(false));
  });
  if (attr != cudaSuccess) return attr;
  const int groups = (a.m + a.nodes_per_tile - 1) / a.nodes_per_tile;
  const int tiles = (a.C + NT - 1) / NT;
  const long long units = static_cast<long long>(a.B) * a.Hkv * groups;
  // one wave: a second one would pay the set-up and the queries' rounding again
  const int gx = static_cast<int>(std::min<long long>(tiles, std::max<long long>(1, num_sms / units)));
  return launch_pdl(score_kernel<T, NCH, NT>, dim3(gx, groups, a.B * a.Hkv), dim3(kScoreThreads), C::bytes(a.lg >= 0), stream,
                    a);
}

template <typename T>
cudaError_t launch_score(const SelectArgs& a, cudaStream_t stream, int num_sms) {
  // 128 pages a tile while the operands leave room for four stages of half a tile, else 64 pages and two stages
  if (a.d <= 64) return launch_score<T, 1, 128>(a, stream, num_sms);
  return a.d <= 128 ? launch_score<T, 2, 128>(a, stream, num_sms) : launch_score<T, 4, 64>(a, stream, num_sms);
}

int score_stride(int C) { return (C + 127) / 128 * 128; }

size_t scores_bytes(int B, int m, int Hkv, int C) { return static_cast<size_t>(B) * Hkv * m * score_stride(C) * 4; }

}  // namespace

size_t page_select_workspace_bytes(int B, int m, int Hq, int Hkv, int d, int C) {
  if (one_node(B, m, Hq, Hkv, d, C)) return 256;
  return scores_bytes(B, m, Hkv, C) + static_cast<size_t>(B) * Hkv * C * ((m + 63) / 64) * 8;
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
  a.stride = score_stride(a.C);
  a.lg = fold_by_shuffles(a.g) ? 31 - __builtin_clz(static_cast<unsigned>(a.g)) : -1;
  a.q_vec = c.d % 8 == 0 && (reinterpret_cast<uintptr_t>(c.q) & 15u) == 0;
  a.scores = static_cast<float*>(c.workspace);
  a.dense = reinterpret_cast<unsigned long long*>(static_cast<char*>(c.workspace) + scores_bytes(c.B, c.m, c.Hkv, a.C));
  if (one_node(c.B, c.m, c.Hq, c.Hkv, c.d, a.C)) {
    count_launches(1);
    return (c.dt == TS_BF16 ? launch_one<__nv_bfloat16>(a, stream) : launch_one<float>(a, stream)) == cudaSuccess ? TS_OK
                                                                                                              : TS_ERR_CUDA;
  }
  cudaError_t e = c.dt == TS_BF16 ? launch_score<__nv_bfloat16>(a, stream, num_sms) : launch_score<float>(a, stream, num_sms);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  const long long rows = static_cast<long long>(c.B) * c.Hkv * c.m;
  const int wpc = kChooseWarpThreads / 32;
  const dim3 warps(static_cast<unsigned>((rows + wpc - 1) / wpc)), wblock(kChooseWarpThreads);
  const dim3 ctas(static_cast<unsigned>(rows)), block(kChooseThreads);
  if (a.C <= 2048) {
    const bool one = c.m == 1;
    auto* choose = a.C <= 512 ? (one ? choose_warp_kernel<16, true> : choose_warp_kernel<16, false>)
                   : a.C <= 1024 ? (one ? choose_warp_kernel<32, true> : choose_warp_kernel<32, false>)
                                 : (one ? choose_warp_kernel<64, true> : choose_warp_kernel<64, false>);
    e = launch_pdl(choose, warps, wblock, 0, stream, a, rows);
    if (one) {
      count_launches(1);
      return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
    }
  } else if (a.C <= 32 * kChooseThreads) {
    e = launch_pdl(choose_kernel<32>, ctas, block, 0, stream, a);
  } else {
    e = launch_pdl(choose_kernel<0>, ctas, block, 0, stream, a);
  }
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  e = launch_pdl(pack_kernel, dim3(c.B * c.Hkv), dim3(kPackThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  return TS_OK;
}

}  // namespace ts
