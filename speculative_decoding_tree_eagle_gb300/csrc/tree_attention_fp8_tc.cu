// ts_tree_attention_fp8, tensor-core path (bf16 queries, head dim 128, pages of 16, 32, 64 or 128 tokens) for sm_103a.
//
// Mathematics.  Rows are (node, head of the KV head's group); key j has codes K_j, V_j (e4m3) and scales ks_j, vs_j:
//   y_ij = (q_i . K_j) * ks_j * scale * log2 e + log2 vs_j
//   M_i  = a running reference of y_i,  p'_ij = 2^(y_ij - M_i)
//   out_i = sum_j p'_ij V_j / sum_j p'_ij / vs_j,    lse_i = ln 2 * (M_i + log2 sum_j p'_ij / vs_j)
// V's scale goes into the exponent, so the reference is that of the contributions p * v, not of the weights p alone: what
// is small against it is small in the output, whatever the scales are.
//
// Layout.  The products are transposed, keys (then channels) in the 128 rows of the tensor-core tile and the queries'
// R rows (16, 32, 64 or 128) in its columns:
//   S^T [128 keys x R]     = K (8 bits, as it lies in the cache) x Q^T
//   O^T [128 channels x R] += V^T (fp16) x P^T (fp16)
// A thread of the softmax then has one key (its TMEM lane): its scales are two registers, and a call with few rows computes
// few columns instead of 128 rows of padding, which is what single tokens and chains need (a 128-key tile's bytes
// take some 1400 cycles of an SM's share of the HBM, less than the softmax of 128 x 128 scores).
//   Q   each row is scaled by a power of two of its own to at most 256 and split into e4m3 + e5m2: a bf16 value has eight
//       significant bits, the nearest e4m3 takes four and leaves a remainder of at most three, which e5m2 holds; what falls
//       below 2^-25 of the row's largest value is lost.  Two MMAs of kind f8f6f4 (twice fp16's rate) on the
//       codes replace a conversion of K.
//   V   is converted to fp16 in shared memory (exact) by warps of their own: weights of eight bits would need the product
//       three times over.
//   P'  is rounded to fp16 (half a step of 2^-11, nothing lost above 2^-25 / 2^7 of the reference): M is kept 7 below the
//       largest y and is raised only when a y exceeds it by 15, so p' <= 2^15.  The sum is of the unrounded p', in fp32.
//
// Work.  One CTA per SM walks an even share of the tiles of all (sequence, KV head) units, R rows of them at a time: a
// run may begin and end inside a unit.  Units that one CTA has whole are written at once, the parts of the others go
// to the workspace and join_kernel merges them.  With several row groups CTAs of neighbouring index walk the same tiles
// for different rows, so all but one read them from L2.
//
// Warps: 0 TMA copies of K, 1 K Q^T and owner of the tensor memory, 2 scales, 3 copies of V, 4..7 Q and V converters, 8 and 9 second
// ones of 0 and 3, 10 idle, 11 V^T P^T, from 12 on softmax: four warps (one per 32 TMEM lanes) for every CPT columns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "fp8_cache.cuh"
#include "internal.h"

namespace ts {
namespace fp8tc {

constexpr int HD = 128;
constexpr int BK = 128;                      // keys per tile
constexpr uint32_t TILE8 = BK * HD;          // codes of one tile of K or V
constexpr uint32_t TILE16 = 2 * TILE8;       // V in fp16
constexpr int kScaleSlots = 4;
constexpr float kFloor = -1e30f;             // reference of a row that has met no key
constexpr float kBelow = 7.f, kRise = 15.f;  // the reference lies kBelow under the largest y; raised when exceeded by kRise
constexpr float kLn2f = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634074f;

template <int R>
struct Cfg {
  static constexpr int CPT = R == 16 ? 16 : R == 32 ? 16 : 32;  // columns per softmax thread
  static constexpr int NG = R / CPT;                             // column groups of four warps
  static constexpr int SOFT = 4 * NG;
  // A TMA copy keeps its issuing warp busy for some 140 cycles and a tile of 16-token pages is 16 of them: up to 64 rows, where
  // a tile has to be done in the time that its bytes take, K and V have two issuing warps each.
  static constexpr int EXTRA = 4;
  static constexpr int ISSUERS = R == 128 ? 1 : 2;
  static constexpr int FIRST_SOFT = 8 + EXTRA;
  static constexpr int THREADS = 32 * (FIRST_SOFT + SOFT);
  static constexpr int SK = R == 128 ? 3 : R == 16 ? 5 : 4;
  static constexpr int SV = R >= 64 ? 2 : 4;
  static constexpr int NP = R == 128 ? 1 : 2;                    // P buffers
  static constexpr int NV = 2;                                   // fp16 V buffers
  static constexpr uint32_t PROW = R >= 64 ? 128 : 2 * R;        // bytes of a P row inside a swizzle atom
  static constexpr uint32_t QPART = R * HD;                      // one of Q's two parts
  static constexpr uint32_t PBUF = BK * R * 2;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * QPART;
  static constexpr uint32_t OFF_V = OFF_K + SK * TILE8;
  static constexpr uint32_t OFF_V16 = OFF_V + SV * TILE8;
  static constexpr uint32_t OFF_P = OFF_V16 + NV * TILE16;
  static constexpr uint32_t OFF_SC = OFF_P + NP * PBUF;          // {ks * scale * log2 e, log2 vs} per key
  static constexpr uint32_t OFF_RM = OFF_SC + kScaleSlots * BK * 8;  // per pair of rows {r0, r1, -M0, -M1}
  static constexpr uint32_t OFF_R2 = OFF_RM + R * 8;             // row scales of the next segment
  static constexpr uint32_t OFF_RED = OFF_R2 + R * 4;            // [4 quarters][R]
  static constexpr uint32_t OFF_FAC = OFF_RED + 4 * R * 4;       // [R]
  static constexpr uint32_t OFF_BAR = OFF_FAC + R * 4;
  static constexpr int NBAR = 2 * SK + 2 * SV + 2 * NV + 4 + 2 * NP + 2 * kScaleSlots + 5;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t SMEM = OFF_MISC + 64 + 1024;
  static constexpr uint32_t TMEM_COLS = R == 16 ? 64 : 4 * R;    // O, S_0, S_1 (a power of two)
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct Params {
  const __nv_bfloat16* q;
  const float* ks;
  const float* vs;
  const uint8_t* vc;
  const int32_t* table;
  const int32_t* prefix_len;
  const uint64_t* mask;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;    // [RG * Gr, 2, R, 128]
  float2* part_ml;  // [RG * Gr, 2, R]
  int32_t* status;
  int B, m, Hq, Hkv, g, rows, W, bs, nsb, bs_log2, sb_log2, max_blocks, num_blocks, max_prefix;
  int RG, Gr;       // row groups, CTAs per row group
  float scale_log2;
};

__device__ __forceinline__ int tiles_of(const Params& p, int b) {
  const int L = p.prefix_len[b];
  if (L < 0 || L > p.max_prefix || static_cast<long long>(L) + p.m > static_cast<long long>(p.max_blocks) * p.bs) return 0;
  return (L + p.m + BK - 1) / BK;
}

// A run of tiles of one unit.
struct Segment {
  int b, h, t0, t1, T, L;
};
// The segments of the tile range [x, x1), from sequence b on; `off` tiles into its unit h.
struct Walk {
  long long x, x1;
  int b, h, off;
  __device__ __forceinline__ bool next(const Params& p, Segment& s) {
    if (x >= x1) return false;
    int T = tiles_of(p, b);
    while (T == 0) {  // (x < x1: a sequence with tiles follows)
      ++b;
      T = tiles_of(p, b);
    }
    s.b = b, s.h = h, s.T = T, s.L = p.prefix_len[b];
    s.t0 = off;
    s.t1 = static_cast<int>(min(static_cast<long long>(T), off + (x1 - x)));
    x += s.t1 - s.t0;
    off = s.t1;
    if (off == T) {
      off = 0;
      if (++h == p.Hkv) h = 0, ++b;
    }
    return true;
  }
};

// All tiles of a row group, and where tile x lies (by one warp).
__device__ __forceinline__ long long total_tiles(const Params& p, int lane) {
  long long n = 0;
  for (int b = lane; b < p.B; b += 32) n += tiles_of(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * p.Hkv;
}
__device__ __forceinline__ Walk walk_from(const Params& p, long long x, long long x1, int lane) {
  Walk w{x, x1, 0, 0, 0};
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int T = b0 + lane < p.B ? tiles_of(p, b0 + lane) : 0;
    long long sum = static_cast<long long>(T) * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + sum > x);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      const int Tl = __shfl_sync(0xffffffffu, T, l);
      const long long at = x - (before + __shfl_sync(0xffffffffu, sum, l) - static_cast<long long>(Tl) * p.Hkv);
      w.b = b0 + l;
      w.h = static_cast<int>(at / Tl);
      w.off = static_cast<int>(at - static_cast<long long>(w.h) * Tl);
      return w;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return w;
}

// The CTA of a row group whose range [c N / Gr, (c + 1) N / Gr) holds tile x (Gr <= N).
__device__ __forceinline__ int cta_of(long long x, long long N, long long Gr) {
  return static_cast<int>(((x + 1) * Gr + N - 1) / N) - 1;
}

__device__ __forceinline__ int block_at(const Params& p, int b, int lp, int pages) {
  if (lp >= pages) return -2;  // behind the sequence: not read
  const int id = __ldg(p.table + static_cast<long long>(b) * p.max_blocks + lp);
  return id >= 0 && id < p.num_blocks ? id : -1;
}

// D (+)= A * B by one lane of a converged warp: 8-bit types, and fp16.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, one;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, one;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The barrier gets an arrival when the MMAs that the elected lane has issued are done.
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
      "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// One box of a tensor map by the elected lane.
__device__ __forceinline__ void tma_elected(uint32_t dst, const void* tmap, uint32_t bar, int c2, int c3) {
  asm volatile(
      "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
      "@one cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// Instruction descriptors (fields as in idesc_bf16_f32; format 0 is e4m3 in kind f8f6f4 and fp16 in kind f16, 1 is e5m2).
__host__ __device__ constexpr uint32_t idesc_of(int N, int b_format, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_format) << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(BK >> 4) << 24);
}
// Shared-memory descriptor with a swizzle of `row` bytes (128, 64 or 32): layout codes 2, 4, 6.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t row) {
  const uint64_t layout = row == 128 ? 2 : row == 64 ? 4 : 6;
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (layout << 61);
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
// 16 consecutive columns of this thread's lane, and wait for them.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : TS_R8(0), TS_R8(8)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      TS_W8(0), TS_W8(8)
      : "memory");
}

// Named barriers of the softmax's column groups: 128 threads each.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + group), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0u;
}
// Floats as integers of the same order (no NaN).
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// Bounded wait of a whole warp.  Every branch on its way is a vote, so what follows is uniform to the compiler too: descriptors and
// addresses of MMAs and copies then stay in uniform registers instead of being moved there for each instruction, which
// took some 100 cycles an MMA and 140 a copy where one lane issued them.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    if ((it & 63u) == 0u) {
      const bool late = global_timer_ns() - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, *abort_flag != 0 || late)) {
        if (late && (threadIdx.x & 31) == 0 && *abort_flag == 0) {
          *abort_flag = 1;
          report(status, TS_ERR_TIMEOUT);
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, late)) *abort_flag = 1;
        return false;
      }
    }
  }
}

// On the way out after a failed wait: lets copies and MMAs in flight land.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
  }
}

// Sums of each of N columns over a warp's lanes: lane c (mod N) ends with column c's.
template <int N>
__device__ __forceinline__ float column_sums(float (&v)[N], int lane) {
  int width = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (width > 1 && o < N) {
      width >>= 1;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < width) {
          const bool up = (lane & o) != 0;
          const float mine = up ? v[i + width] : v[i], theirs = up ? v[i] : v[i + width];
          v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
        }
      }
    } else {
      // (N = 16: lanes 16 apart hold the same columns)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < width) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
  return v[0];
}

template <int R>
__global__ void __launch_bounds__(Cfg<R>::THREADS, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const __grid_constant__ Params p) {
  using C = Cfg<R>;
  constexpr int HALF = 16;  // columns that a softmax thread works on at a time
  constexpr int CPT = C::CPT, SK = C::SK, SV = C::SV, NP = C::NP, NV = C::NV;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sptr = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = blockIdx.x % p.RG, cta = blockIdx.x / p.RG;
  const int R0 = rg * R, rows_here = min(R, p.rows - R0);

  uint32_t at = sbase + C::OFF_BAR;
  auto take = [&](int n) {
    const uint32_t first = at;
    at += 8u * n;
    return first;
  };
  const uint32_t full_k = take(SK), empty_k = take(SK), full_v = take(SV), empty_v = take(SV), v16_full = take(NV),
                 v16_empty = take(NV), s_full = take(2), s_empty = take(2), p_full = take(NP), p_empty = take(NP),
                 sc_full = take(kScaleSlots), sc_empty = take(kScaleSlots), q_full = take(1),
                 q_empty = take(1), o_free = take(1), last = take(2);
  unsigned char* misc = sptr + C::OFF_MISC;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* nan_seg = reinterpret_cast<volatile int*>(misc + 8);  // [2]: the segment (+1) whose tree rows have NaN in V
  Walk* s_walk = reinterpret_cast<Walk*>(misc + 16);

  if (threadIdx.x == 0) {
    for (int i = 0; i < SK; ++i) mbar_init(full_k + 8 * i, C::ISSUERS), mbar_init(empty_k + 8 * i, 1);
    for (int i = 0; i < SV; ++i) mbar_init(full_v + 8 * i, C::ISSUERS), mbar_init(empty_v + 8 * i, 4);
    for (int i = 0; i < NV; ++i) mbar_init(v16_full + 8 * i, 4), mbar_init(v16_empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(s_full + 8 * i, 1), mbar_init(s_empty + 8 * i, C::SOFT);
    for (int i = 0; i < NP; ++i) mbar_init(p_full + 8 * i, C::SOFT), mbar_init(p_empty + 8 * i, 1);
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(sc_full + 8 * i, 1), mbar_init(sc_empty + 8 * i, C::SOFT);
    mbar_init(q_full, 4);
    mbar_init(q_empty, 1 + C::SOFT);
    mbar_init(last, 1);
    mbar_init(last + 8, 1);
    mbar_init(o_free, C::SOFT);
    *abort_flag = 0;
    nan_seg[0] = nan_seg[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 0) {
    const long long N = total_tiles(p, lane);
    const long long Gr = min(static_cast<long long>(p.Gr), N);  // (no CTA between two parts of a unit is without tiles)
    const Walk w = cta < Gr ? walk_from(p, cta * N / Gr, (cta + 1) * N / Gr, lane) : Walk{0, 0, 0, 0, 0};
    if (lane == 0) *s_walk = w;
    if (blockIdx.x == 0)
      for (int b = lane; b < p.B; b += 32)
        if (tiles_of(p, b) == 0) report(p.status, TS_ERR_DEVICE_CHECK);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  Walk walk = *s_walk;
  Segment sg;
  const int ppt = BK >> p.bs_log2;  // pages per tile
  bool ok = true;

  // warps 8..11: second issuers of K and V, the second scale warp, and P V
  const int part = warp >= 8 && warp < 11 ? 1 : 0;
  const int role = warp < 4 ? warp : warp < 8 ? 5 : warp == 11 ? 4 : warp >= C::FIRST_SOFT ? 6 : C::ISSUERS == 1 || warp == 10 ? -1 : warp == 8 ? 0 : 3;
  if (role == 0 || role == 3) {
    // ------------------------------ codes by TMA (role 0: K, 3: V): lane i issues page ISSUERS i + part of a tile ------------------------------
    const bool is_k = role == 0;
    const int stages = is_k ? SK : SV;
    const uint32_t full = is_k ? full_k : full_v, empty = is_k ? empty_k : empty_v;
    const uint32_t ring = sbase + (is_k ? C::OFF_K : C::OFF_V);
    const CUtensorMap* map = is_k ? &tmk : &tmv;
    const int my = C::ISSUERS * lane + part;
    const int mine = (ppt + C::ISSUERS - 1 - part) / C::ISSUERS;  // pages of a tile that this warp issues
    const bool issues = my < ppt;
    int it = 0, stage = 0, phase = 0;
    while (ok && walk.next(p, sg)) {
      const int pages = (sg.L + p.m + p.bs - 1) >> p.bs_log2;
      int id = issues ? block_at(p, sg.b, sg.t0 * ppt + my, pages) : 0;
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int cur = id;
        if (issues && t + 1 < sg.t1) id = block_at(p, sg.b, (t + 1) * ppt + my, pages);
        if (cur == -1) report(p.status, TS_ERR_DEVICE_CHECK);
        const int blk = cur < 0 ? p.num_blocks : cur;  // (out of range: the copy fills zeros)
        ok = wait_warp(empty + 8 * stage, phase ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full + 8 * stage, mine * p.bs * HD);
        __syncwarp();
        for (int i = 0; i < mine; ++i)
          tma_elected(ring + stage * TILE8 + (C::ISSUERS * i + part) * p.bs * HD, map, full + 8 * stage, sg.h,
                      __shfl_sync(0xffffffffu, blk, i));
        if (++stage == stages) stage = 0, phase ^= 1;
      }
    }
    // after an abort nobody waits for what is still on its way: the newest copy of every stage
    if (!ok)
      for (int i = max(0, it - stages); i < it; ++i) drain(full + 8 * (i % stages), (i / stages) & 1);
  } else if (role == 1) {
    // ------------------------------ S^T = K Q^T (the warp issues as one) ------------------------------
    constexpr uint32_t iq1 = idesc_of(R, 0, 0, 0), iq2 = idesc_of(R, 1, 0, 0);
    const uint64_t kdesc = sdesc(sbase + C::OFF_K, 16, 1024, 128), qdesc = sdesc(sbase + C::OFF_Q, 16, 1024, 128);
    int it = 0, seg = 0;
    while (ok && walk.next(p, sg)) {
      ok = wait_warp(q_full, seg & 1, abort_flag, p.status);
      if (!ok) break;
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int sk = it % SK, s = it & 1;
        ok = wait_warp(full_k + 8 * sk, (it / SK) & 1, abort_flag, p.status);
        if (!ok) break;
        ok = wait_warp(s_empty + 8 * s, ((it >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + R + R * s;
        // (descriptors count 16-byte units: a step of 32 bytes adds 2)
        const uint64_t kd = kdesc + static_cast<uint64_t>(sk * (TILE8 >> 4));
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk) mma_f8(d, kd + 2u * kk, qdesc + 2u * kk, iq1, kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk) mma_f8(d, kd + 2u * kk, qdesc + (C::QPART >> 4) + 2u * kk, iq2, 1u);
        commit_elected(s_full + 8 * s);
        commit_elected(empty_k + 8 * sk);
      }
      if (!ok) break;
      commit_elected(q_empty);
      ++seg;
    }
    if (!ok) {
      // MMAs in flight end before the accumulators are given back
      commit_elected(last);
      drain(last, 0);
    }
  } else if (role == 4) {
    // ------------------------------ O^T += V^T P^T ------------------------------
    constexpr uint32_t ip = idesc_of(R, 0, 1, 1);
    const uint64_t vdesc = sdesc(sbase + C::OFF_V16, BK * 128, 1024, 128);
    const uint64_t pdesc = sdesc(sbase + C::OFF_P, BK * 128, 8 * C::PROW, C::PROW);
    int it = 0, seg = 0;
    while (ok && walk.next(p, sg)) {
      // (the accumulator is free once the last segment's has been read)
      ok = wait_warp(o_free, (seg & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int v = it % NV, pb = it % NP;
        ok = wait_warp(v16_full + 8 * v, (it / NV) & 1, abort_flag, p.status);
        if (!ok) break;
        ok = wait_warp(p_full + 8 * pb, (it / NP) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vdesc + static_cast<uint64_t>(v * (TILE16 >> 4)), pd = pdesc + static_cast<uint64_t>(pb * (C::PBUF >> 4));
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_f16(tmem, vd + (2048u >> 4) * kk, pd + C::PROW * kk, ip, kk > 0 || t > sg.t0 ? 1u : 0u);
        commit_elected(v16_empty + 8 * v);
        commit_elected(p_empty + 8 * pb);
      }
      ++seg;
    }
    if (!ok) {
      commit_elected(last + 8);
      drain(last + 8, 0);
    }
  } else if (role == 2) {
    // ------------------------------ scales ------------------------------
    // Four tiles' scales are under way in registers, and the ids of the next four: one tile ahead the two dependent loads set the
    // pace (4800 cycles a tile unprefetched, 1700 one ahead, where a tile's bytes take 1400).
    constexpr int AHEAD = 4;
    int it = 0;
    while (ok && walk.next(p, sg)) {
      const int pages = (sg.L + p.m + p.bs - 1) >> p.bs_log2, n = sg.t1 - sg.t0;
      int id[AHEAD][4];
      float ks[AHEAD][4], vs[AHEAD][4];
      bool id_was[AHEAD][4];
      auto ids = [&](int u, int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) id[u][j] = i < n ? block_at(p, sg.b, ((sg.t0 + i) * BK + 32 * j + lane) >> p.bs_log2, pages) : -2;
      };
      auto load = [&](int u, int i) {  // with the ids of tile i; a page without an id: its keys get no weight
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ks[u][j] = 0.f, vs[u][j] = 0.f;
          id_was[u][j] = id[u][j] >= 0;
          if (id_was[u][j]) {
            const int row = ((sg.t0 + i) * BK + 32 * j + lane) & (p.bs - 1);
            const long long o = (static_cast<long long>(id[u][j]) * p.Hkv + sg.h) * p.nsb + (row >> p.sb_log2);
            ks[u][j] = __ldg(p.ks + o);
            vs[u][j] = __ldg(p.vs + o);
          }
        }
      };
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) ids(u, u);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) load(u, u);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) ids(u, AHEAD + u);
      for (int i = 0; ok && i < n; i += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (!ok || i + u >= n) break;
          const int slot = (it + u) % kScaleSlots;
          ok = wait_warp(sc_empty + 8 * slot, (((it + u) / kScaleSlots) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          float2* to = reinterpret_cast<float2*>(sptr + C::OFF_SC) + slot * BK;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            to[32 * j + lane] = make_float2(scale_in_range(ks[u][j]) * p.scale_log2,
                                            id_was[u][j] ? __log2f(scale_in_range(vs[u][j])) : -INFINITY);
          __syncwarp();
          if (lane == 0) mbar_arrive(sc_full + 8 * slot);
        }
        it += min(AHEAD, n - i);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) load(u, i + AHEAD + u);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) ids(u, i + 2 * AHEAD + u);
      }
    }
  } else if (role == 5) {
    // ------------------------------ Q and V into the tensor cores' types ------------------------------
    const int w = warp - 4;
    int it = 0, seg = 0;
    while (ok && walk.next(p, sg)) {
      ok = wait_warp(q_empty, (seg & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
      // eight lanes per row, 16 values each
      for (int r0 = w * 4; r0 < R; r0 += 16) {
        const int r = r0 + (lane >> 3), c = lane & 7;
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (r < rows_here) {
          const int row = R0 + r, node = row / p.g, head = sg.h * p.g + row % p.g;
          const uint4* src = reinterpret_cast<const uint4*>(p.q + ((static_cast<long long>(sg.b) * p.m + node) * p.Hq + head) * HD) + 2 * c;
          x[0] = __ldg(src);
          x[1] = __ldg(src + 1);
        }
        const uint32_t in[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
        float v[16];
        uint32_t big = 0;  // largest magnitude, as bits (an infinity or a NaN makes the row NaN)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[2 * j] = bf16_lo(in[j]);
          v[2 * j + 1] = bf16_hi(in[j]);
          big = max(big, max(__float_as_uint(v[2 * j]) & 0x7FFFFFFFu, __float_as_uint(v[2 * j + 1]) & 0x7FFFFFFFu));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        // 2^e: the largest magnitude times 2^-e lies in [128, 256) (2^-e in two factors, as it may pass 2^127)
        const int e = static_cast<int>(big >> 23) - 127 - 7;
        const float f0 = pow2(-(e / 2)), f1 = pow2(-(e - e / 2));
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a = 0, b2 = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float y0 = v[4 * j + 2 * u] * f0 * f1, y1 = v[4 * j + 2 * u + 1] * f0 * f1;
            const uint32_t two = encode_e4m3x2(y0, y1);
            const float2 back = decode_e4m3x2(two);
            a |= two << (16 * u);
            b2 |= encode_e5m2x2(y0 - back.x, y1 - back.y) << (16 * u);
          }
          hi[j] = a, lo[j] = b2;
        }
        const uint32_t off = r * 128 + ((c ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(sptr + C::OFF_Q + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sptr + C::OFF_Q + C::QPART + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (c == 0) reinterpret_cast<float*>(sptr + C::OFF_R2)[r] = big >= 0x7F800000u ? __int_as_float(0x7FC00000) : pow2(max(-126, e));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int sv = it % SV, v = it % NV;
        ok = wait_warp(full_v + 8 * sv, (it / SV) & 1, abort_flag, p.status) &&
             wait_warp(v16_empty + 8 * v, ((it / NV) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        const unsigned char* from = sptr + C::OFF_V + sv * TILE8;
        unsigned char* to = sptr + C::OFF_V16 + v * TILE16;
        const bool tail = (t + 1) * BK > sg.L;
        // Keys in groups of eight; of a group, lanes of one eighth of the warp take keys k and k ^ 5 and four 16-byte chunks:
        // reads (chunk c at c ^ (k % 8)) and writes (chunks 2c, 2c + 1 of the half's 128-byte row, the same way) then touch
        // all banks once.
        const int pair = lane >> 3, k8 = (lane & 4) ? pair ^ 5 : pair, c4 = lane & 3;
        // (all loads first: with a branch and a store between them each waited for its own, 2400 cycles a tile)
        uint4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          x[u] = *reinterpret_cast<const uint4*>(from + ((w * 4 + (u >> 1)) * 8 + k8) * 128 + (((c4 + 4 * (u & 1)) ^ k8) << 4));
        if (tail) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int pos = t * BK + (w * 4 + (u >> 1)) * 8 + k8;
            if (pos >= sg.L + p.m) {
              x[u] = make_uint4(0, 0, 0, 0);
            } else if (pos >= sg.L) {
              // a NaN of a tree row reaches the rows that attend to it in the epilogue: here it would reach all
              const uint32_t n0 = __vcmpeq4(x[u].x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), n1 = __vcmpeq4(x[u].y & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                             n2 = __vcmpeq4(x[u].z & 0x7F7F7F7Fu, 0x7F7F7F7Fu), n3 = __vcmpeq4(x[u].w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              if ((n0 | n1 | n2 | n3) != 0u) {
                nan_seg[seg & 1] = seg + 1;
                x[u] = make_uint4(x[u].x & ~n0, x[u].y & ~n1, x[u].z & ~n2, x[u].w & ~n3);
              }
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          unsigned char* row = to + (u & 1) * (BK * 128) + ((w * 4 + (u >> 1)) * 8 + k8) * 128;
          *reinterpret_cast<uint4*>(row + (((2 * c4) ^ k8) << 4)) =
              make_uint4(decode_e4m3x2_f16(x[u].x), decode_e4m3x2_f16(x[u].x >> 16), decode_e4m3x2_f16(x[u].y),
                         decode_e4m3x2_f16(x[u].y >> 16));
          *reinterpret_cast<uint4*>(row + (((2 * c4 + 1) ^ k8) << 4)) =
              make_uint4(decode_e4m3x2_f16(x[u].z), decode_e4m3x2_f16(x[u].z >> 16), decode_e4m3x2_f16(x[u].w),
                         decode_e4m3x2_f16(x[u].w >> 16));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(empty_v + 8 * sv);
          mbar_arrive(v16_full + 8 * v);
        }
      }
      ++seg;
    }
  } else if (role == 6) {
    // ------------------------------ softmax ------------------------------
    const int quarter = warp & 3, group = (warp - C::FIRST_SOFT) >> 2, col0 = group * CPT;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    float4* rm = reinterpret_cast<float4*>(sptr + C::OFF_RM) + col0 / 2;  // {r0, r1, -M0, -M1} of this group's pairs
    float* rmf = reinterpret_cast<float*>(rm);
    float* red = reinterpret_cast<float*>(sptr + C::OFF_RED) + col0;      // [quarter * R + c]
    float* fac = reinterpret_cast<float*>(sptr + C::OFF_FAC) + col0;
    // P V of tile i is done: its P buffer is free again.  (A barrier of one phase per tile would not do: with two P buffers
    // the softmax may be two tiles ahead of P V, and a wait by parity would take the older phase for the newer.)
    auto o_holds = [&](int i) { return wait_warp(p_empty + 8 * (i % NP), (i / NP) & 1, abort_flag, p.status); };
    auto m_at = [&](int c) -> float& { return rmf[(c >> 1) * 4 + 2 + (c & 1)]; };
    int it = 0, seg = 0;
    while (walk.next(p, sg)) {
      if (ok) ok = wait_warp(q_full, seg & 1, abort_flag, p.status);
      if (group_any(group, !ok)) {
        ok = false;
        break;
      }
      if (quarter == 0 && lane < CPT) {
        rmf[(lane >> 1) * 4 + (lane & 1)] = reinterpret_cast<const float*>(sptr + C::OFF_R2)[col0 + lane];
        m_at(lane) = col0 + lane < rows_here ? -kFloor : kFloor;  // (padding: weights 0)
      }
      group_sync(group);
      if (lane == 0) mbar_arrive(q_empty);  // (the row scales are taken; the MMA thread says when Q is)
      uint64_t l2[CPT / 2];
#pragma unroll
      for (int c = 0; c < CPT / 2; ++c) l2[c] = 0ull;
      // {r0, r1, -M0, -M1}: with 16 columns they stay in registers
      float4 held[HALF / 2];
      auto hold = [&]() {
        if (CPT == HALF) {
#pragma unroll
          for (int c = 0; c < HALF / 2; ++c) held[c] = rm[c];
        }
      };
      hold();
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int s = it & 1, slot = it % kScaleSlots;
        const uint32_t tS = tmem + lanes + R + R * s + col0;
        if (ok)
          ok = wait_warp(sc_full + 8 * slot, (it / kScaleSlots) & 1, abort_flag, p.status) &&
               wait_warp(s_full + 8 * s, (it >> 1) & 1, abort_flag, p.status);
        float2 sc = make_float2(0.f, 0.f);
        uint32_t x[HALF];
        float zmax = -INFINITY;
        const bool tail = (t + 1) * BK > sg.L;
        uint32_t vis = 0u;  // bit c: row c attends to this key (tail tiles)
        auto scores = [&](int half) {  // x <- z = y - M of 16 columns
          tmem_ld(tS + HALF * half, x);
          const uint64_t a2 = pack_f32x2(sc.x, sc.x), v2 = pack_f32x2(sc.y, sc.y);
#pragma unroll
          for (int c = 0; c < HALF; c += 2) {
            const float4 k = CPT == HALF ? held[c / 2] : rm[(HALF * half + c) / 2];
            const uint64_t z2 = fma_f32x2(pack_f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                          mul_f32x2(a2, pack_f32x2(k.x, k.y)), add_f32x2(v2, pack_f32x2(k.z, k.w)));
            float z0, z1;
            unpack_f32x2(z2, z0, z1);
            x[c] = __float_as_uint(z0);
            x[c + 1] = __float_as_uint(z1);
          }
          if (tail) {
#pragma unroll
            for (int c = 0; c < HALF; ++c)
              if (!((vis >> (HALF * half + c)) & 1u)) x[c] = 0xFF800000u;
          }
        };
        auto highest = [&]() {
#pragma unroll
          for (int c = 0; c < HALF; c += 2) zmax = max3(zmax, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        };
        if (ok) {
          tc_fence_after();
          sc = reinterpret_cast<const float2*>(sptr + C::OFF_SC)[slot * BK + 32 * quarter + lane];
          if (tail) {
            // which of this thread's rows attend to its key
            const int n = t * BK + 32 * quarter + lane - sg.L;
            vis = sc.y == -INFINITY ? 0u : ~0u;
            if (n >= p.m) vis = 0u;
            const int word = min(max(n, 0), p.m - 1) >> 6;
            uint32_t seen = 0u;
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
              const int row = min(R0 + col0 + c, p.rows - 1);
              const uint64_t w = __ldg(p.mask + (static_cast<long long>(sg.b) * p.m + row / p.g) * p.W + word);
              seen |= static_cast<uint32_t>((w >> (n & 63)) & 1ull) << c;
            }
            if (n >= 0) vis &= seen;
          }
          // The first pass finds whether the reference has to rise, the second makes the weights; between them 32 columns'
          // scores stay in tensor memory (kept in registers beside the sums they spilled: 7500 cycles a tile of 128 rows).
#pragma unroll
          for (int half = 0; half < CPT / HALF; ++half) {
            scores(half);
            highest();
          }
        }
        if (group_any(group, !ok || zmax > kRise)) {
          // Rare: a reference has to rise (every unit's first tile does this).
          if (group_any(group, !ok)) {
            ok = false;
            break;
          }
          int top = 0x80000000;
#pragma unroll
          for (int half = 0; half < CPT / HALF; ++half) {
            tmem_ld(tS + HALF * half, x);
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
              const int c = HALF * half + i;
              const float r = rmf[(c >> 1) * 4 + (c & 1)];
              float y = fmaf(__uint_as_float(x[i]), sc.x * r, sc.y);
              if (y != y || (tail && !((vis >> c) & 1u))) y = -INFINITY;  // (a NaN goes into the weights, not into the reference)
              const int most = __reduce_max_sync(0xffffffffu, ordered(y));
              if (lane == c) top = most;
            }
          }
          if (lane < CPT) red[quarter * R + lane] = from_ordered(top);
          group_sync(group);
          if (quarter == 0 && lane < CPT) {
            const float old = -m_at(lane);
            const float most = fmaxf(fmaxf(red[lane], red[R + lane]), fmaxf(red[2 * R + lane], red[3 * R + lane])) - kBelow;
            const float M = most > old ? most : old;
            fac[lane] = M == old ? 1.f : ex2_approx(old - M);
            m_at(lane) = -M;
          }
          group_sync(group);
#pragma unroll
          for (int c = 0; c < CPT / 2; ++c) l2[c] = mul_f32x2(l2[c], pack_f32x2(fac[2 * c], fac[2 * c + 1]));
          if (t > sg.t0) {
            ok = o_holds(it - 1);
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int half = 0; half < CPT / HALF; ++half) {
                tmem_ld(tmem + lanes + col0 + HALF * half, x);
#pragma unroll
                for (int c = 0; c < HALF; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * fac[HALF * half + c]);
                tmem_st(tmem + lanes + col0 + HALF * half, x);
              }
              tmem_st_wait();
            }
          }
          hold();
          if (CPT == HALF) scores(0);
        }
        const int pb = it % NP;
        if (ok) ok = wait_warp(p_empty + 8 * pb, ((it / NP) & 1) ^ 1, abort_flag, p.status);
        if (!ok) continue;  // (leaves at the next vote)
        const float iv = sc.y == -INFINITY ? 0.f : ex2_approx(-sc.y);
        const uint64_t iv2 = pack_f32x2(iv, iv);
        // P^T [key][row]: rows of PROW bytes, 16-byte chunks swizzled with the key
        const int k = 32 * quarter + lane;
        unsigned char* prow = sptr + C::OFF_P + pb * C::PBUF + (col0 / 64) * (BK * 128) + k * C::PROW;
        const int chunk0 = (col0 % 64) / 8;
        const int swz = C::PROW == 128 ? (k & 7) : C::PROW == 64 ? ((k >> 1) & 3) : ((k >> 2) & 1);
#pragma unroll
        for (int half = 0; half < CPT / HALF; ++half) {
          if (CPT > HALF) scores(half);
          if (half + 1 == CPT / HALF) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(s_empty + 8 * s);
              mbar_arrive(sc_empty + 8 * slot);
            }
          }
          uint32_t h[HALF / 2];
#pragma unroll
          for (int c = 0; c < HALF; c += 2) {
            const float p0 = ex2_approx(__uint_as_float(x[c])), p1 = ex2_approx(__uint_as_float(x[c + 1]));
            uint64_t& l = l2[HALF / 2 * half + c / 2];
            l = fma_f32x2(pack_f32x2(p0, p1), iv2, l);
            h[c / 2] = pack_f16x2(p0, p1);
          }
#pragma unroll
          for (int j = 0; j < HALF / 8; ++j)
            *reinterpret_cast<uint4*>(prow + (((chunk0 + HALF / 8 * half + j) ^ swz) << 4)) =
                make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * pb);
      }
      if (ok) ok = o_holds(it - 1);
      if (group_any(group, !ok)) {
        ok = false;
        break;
      }
      // ------------------------------ the segment's result ------------------------------
      tc_fence_after();
      float lv[CPT];
#pragma unroll
      for (int c = 0; c < CPT / 2; ++c) unpack_f32x2(l2[c], lv[2 * c], lv[2 * c + 1]);
      const float mine = column_sums(lv, lane);  // lane c: column c's sum over this warp's keys
      if (lane < CPT) red[quarter * R + lane] = mine;
      group_sync(group);
      const bool whole = sg.t0 == 0 && sg.t1 == sg.T;
      float l = 0.f, M = 0.f;
      if (lane < CPT) {
        l = (red[lane] + red[R + lane]) + (red[2 * R + lane] + red[3 * R + lane]);
        M = -m_at(lane);
      }
      const int ch = 32 * quarter + lane;
      const long long slot = (static_cast<long long>(rg) * p.Gr + cta) * 2 + (sg.t0 == 0 ? 1 : 0);
      if (lane < CPT && quarter == 0 && col0 + lane < rows_here) {
        const int row = R0 + col0 + lane, node = row / p.g, head = sg.h * p.g + row % p.g;
        if (!whole) p.part_ml[slot * R + col0 + lane] = make_float2(M, l);
        else if (p.lse != nullptr)
          p.lse[(static_cast<long long>(sg.b) * p.m + node) * p.Hq + head] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2f;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int half = 0; half < CPT / HALF; ++half) {
        uint32_t o[HALF];
        tmem_ld(tmem + lanes + col0 + HALF * half, o);
        if (half + 1 == CPT / HALF) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        const int first = col0 + HALF * half;
        if (nan_seg[seg & 1] == seg + 1) {
          // a NaN in a tree row's V: the rows that attend to it get it
          for (int n = max(0, sg.t0 * BK - sg.L); n < min(p.m, sg.t1 * BK - sg.L); ++n) {
            const int pos = sg.L + n, id = p.table[static_cast<long long>(sg.b) * p.max_blocks + (pos >> p.bs_log2)];
            if (id < 0 || id >= p.num_blocks) continue;
            const uint32_t code = p.vc[((static_cast<long long>(id) * p.Hkv + sg.h) * p.bs + (pos & (p.bs - 1))) * HD + ch];
            if ((code & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
            for (int c = 0; c < HALF; ++c) {
              const int row = min(R0 + first + c, p.rows - 1);
              const uint64_t word = __ldg(p.mask + (static_cast<long long>(sg.b) * p.m + row / p.g) * p.W + (n >> 6));
              if ((word >> (n & 63)) & 1ull) o[c] = 0x7FC00000u;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          const float f = __shfl_sync(0xffffffffu, inv, HALF * half + c);
          if (first + c < rows_here) {
            if (whole) {
              const int row = R0 + first + c, node = row / p.g, head = sg.h * p.g + row % p.g;
              p.out[((static_cast<long long>(sg.b) * p.m + node) * p.Hq + head) * HD + ch] =
                  __float2bfloat16_rn(__uint_as_float(o[c]) * f);
            } else {
              p.part_o[(slot * R + first + c) * HD + ch] = __uint_as_float(o[c]);
            }
          }
        }
      }
      group_sync(group);  // (red and the references are written again)
      ++seg;
    }
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// A warp per output row: joins the parts of a unit that several CTAs walked, in the order of the CTAs.
template <int R>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.B) * p.Hkv * p.rows) return;
  const int row = static_cast<int>(item % p.rows), bh = static_cast<int>(item / p.rows), b = bh / p.Hkv, h = bh % p.Hkv;
  const int T = tiles_of(p, b);
  if (T == 0) return;
  long long before = 0, N = 0;  // tiles of the sequences before b, of all
  for (int i = lane; i < p.B; i += 32) {
    const int x = tiles_of(p, i);
    N += x;
    if (i < b) before += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    N += __shfl_xor_sync(0xffffffffu, N, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  N *= p.Hkv;
  const long long first = before * p.Hkv + static_cast<long long>(h) * T;
  const long long Gr = min(static_cast<long long>(p.Gr), N);
  const int c0 = cta_of(first, N, Gr), c1 = cta_of(first + T - 1, N, Gr);
  if (c0 == c1) return;  // (one CTA had the whole unit)
  const int rg = row / R, r = row - rg * R;
  auto slot = [&](int c) { return (((static_cast<long long>(rg) * p.Gr + c) * 2 + (c == c0 ? 1 : 0)) * R + r); };
  float M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.part_ml[slot(c)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float2 ml = p.part_ml[slot(c)];
    const float4 o = *reinterpret_cast<const float4*>(p.part_o + slot(c) * HD + 4 * lane);
    const float f = ml.x == M ? 1.f : ex2_approx(ml.x - M);
    l = fmaf(ml.y, f, l);
    acc.x = fmaf(o.x, f, acc.x), acc.y = fmaf(o.y, f, acc.y), acc.z = fmaf(o.z, f, acc.z), acc.w = fmaf(o.w, f, acc.w);
  }
  const int node = row / p.g, head = h * p.g + row % p.g;
  const long long o = (static_cast<long long>(b) * p.m + node) * p.Hq + head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(p.out + o * HD + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[o] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2f;
}

// ------------------------------------------------------------------------------------------ host
struct Plan {
  int R, RG, Gr;
};
int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}
// R: the smallest tile width that holds all rows, 128 at most.  CTAs: one per SM, of kMinTiles tiles at least.
constexpr int kMinTiles = 2;
Plan plan_of(int B, int m, int Hq, int Hkv, int max_prefix, int num_sms) {
  const int rows = m * (Hq / Hkv);
  Plan pl;
  pl.R = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  pl.RG = (rows + pl.R - 1) / pl.R;
  const long long tiles = (static_cast<long long>(max_prefix) + m + BK - 1) / BK * B * Hkv;
  const long long want = std::max(1LL, tiles / kMinTiles);
  pl.Gr = static_cast<int>(std::min<long long>(std::max(1, num_sms / pl.RG), want));
  return pl;
}

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;
EncodeFn get_encode() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}
// Codes [num_blocks, Hkv, bs, 128]: a box is one head of one page, rows of 128 bytes swizzled over 128 bytes.
bool encode_map(CUtensorMap* map, const void* base, int num_blocks, int Hkv, int bs) {
  const EncodeFn enc = get_encode();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {HD, static_cast<cuuint64_t>(bs), static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[3] = {HD, static_cast<cuuint64_t>(bs) * HD, static_cast<cuuint64_t>(Hkv) * bs * HD};
  const cuuint32_t box[4] = {HD, static_cast<cuuint32_t>(bs), 1u, 1u}, estr[4] = {1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R>
int launch(const Params& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attn_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<R>::SMEM);
  });
  if (e != cudaSuccess) return TS_ERR_CUDA;
  e = launch_pdl(attn_kernel<R>, dim3(p.RG * p.Gr), dim3(Cfg<R>::THREADS), Cfg<R>::SMEM, stream, mk, mv, p);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  int launches = 1;
  if (p.Gr > 1) {
    const long long rows = static_cast<long long>(p.B) * p.Hkv * p.rows;
    e = launch_pdl(join_kernel<R>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, stream, p);
    ++launches;
  }
  count_launches(launches);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace fp8tc

bool attention_fp8_uses_tc(ts_dtype dt, int d, int block_size) {
  return dt == TS_BF16 && d == fp8tc::HD && (block_size == 16 || block_size == 32 || block_size == 64 || block_size == 128);
}

size_t attention_fp8_tc_workspace_bytes(int B, int m, int Hq, int Hkv, int max_prefix, int num_sms) {
  const fp8tc::Plan pl = fp8tc::plan_of(B, m, Hq, Hkv, max_prefix, std::max(1, num_sms));
  if (pl.Gr == 1) return 256;
  return static_cast<size_t>(pl.RG) * pl.Gr * 2 * pl.R * (fp8tc::HD * sizeof(float) + sizeof(float2)) + 256;
}

int attention_fp8_tc_launch(const Fp8AttnCall& a, cudaStream_t stream, int num_sms) {
  using namespace fp8tc;
  const Plan pl = plan_of(a.B, a.m, a.Hq, a.Hkv, a.max_prefix, num_sms);
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.ks = a.k_scale, p.vs = a.v_scale, p.vc = static_cast<const uint8_t*>(a.v_cache);
  p.table = a.block_table, p.prefix_len = a.prefix_len, p.mask = a.mask;
  p.out = static_cast<__nv_bfloat16*>(a.out), p.lse = a.lse, p.status = a.dev_status;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(pl.RG) * pl.Gr * 2 * pl.R * HD);
  p.B = a.B, p.m = a.m, p.Hq = a.Hq, p.Hkv = a.Hkv, p.g = a.Hq / a.Hkv, p.rows = a.m * p.g, p.W = (a.m + 63) / 64;
  p.bs = a.block_size, p.nsb = a.block_size / a.scale_block;
  // (a page of a power of two tokens is cut into powers of two: shifts, as a division takes one warp hundreds of cycles)
  p.bs_log2 = log2_of(a.block_size), p.sb_log2 = log2_of(a.scale_block);
  p.max_blocks = a.max_blocks, p.num_blocks = a.num_blocks, p.max_prefix = a.max_prefix;
  p.RG = pl.RG, p.Gr = pl.Gr;
  p.scale_log2 = a.scale * kLog2e;
  CUtensorMap mk, mv;
  if (!encode_map(&mk, a.k_cache, a.num_blocks, a.Hkv, a.block_size) || !encode_map(&mv, a.v_cache, a.num_blocks, a.Hkv, a.block_size))
    return TS_ERR_CUDA;
  switch (pl.R) {
    case 16: return launch<16>(p, mk, mv, stream);
    case 32: return launch<32>(p, mk, mv, stream);
    case 64: return launch<64>(p, mk, mv, stream);
    default: return launch<128>(p, mk, mv, stream);
  }
}

}  // namespace ts
