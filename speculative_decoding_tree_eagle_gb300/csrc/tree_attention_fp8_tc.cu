// ts_tree_attention_fp8, tensor-core path (bf16 queries, head dim 128, pages of 16, 32, 64 or 128 tokens) for sm_103a.
//
// Mathematics.  Rows are (node, head of the KV head's group); key j has codes K_j, V_j (e4m3) and scales ks_j, vs_j:
//   y_ij = (q_i . K_j) * ks_j * scale * log2 e + log2 vs_j
//   M_i  = a running reference of y_i,  p'_ij = 2^(y_ij - M_i)
//   out_i = sum_j p'_ij V_j / sum_j p'_ij / vs_j,    lse_i = ln 2 * (M_i + log2 sum_j p'_ij / vs_j)
// V's scale goes into the exponent, so the reference is that of the contributions p * v, not of the weights p alone: what
// is small against it is small in the output, whatever the scales are.
//
// Layout.  Up to 32 rows ("narrow", R = 16 or 32) the products are transposed, keys (then channels) in the 128 rows of the
// tensor-core tile and the queries' R rows in its columns:
//   S^T [128 keys x R]     = K (8 bits, as it lies in the cache) x Q^T
//   O^T [128 channels x R] += V^T (fp16) x P^T (fp16, from shared memory)
// A thread of the softmax then has one key (its TMEM lane): its scales are two registers, and a call with few rows computes
// few columns instead of 128 rows of padding, which is what single tokens and chains need (a 128-key tile's bytes
// take some 1400 cycles of an SM's share of the HBM, less than the softmax of 128 x 128 scores).  Above 32 rows ("wide", R = 128)
// S [R x 128 keys] = Q x K and O [R x 128 channels] += P x V with P from tensor memory, two threads to a row.
//   Q   each row is scaled by a power of two of its own to a largest magnitude in [128, 256) and split into e4m3 + e5m2: a bf16
//       value has eight significant bits, the nearest e4m3 takes four and leaves a remainder of at most three, which e5m2 holds.
//       That is exact down to e4m3's least normal value, 2^-6; below, e4m3's steps are 2^-9 and the remainder may need up to five
//       bits: it is off by at most 2^-14, 2^-21 of the row's largest, in elements of less than 2^-13 of it.  Two MMAs of kind f8f6f4
//       (twice fp16's rate) on the codes replace a conversion of K.
//   V   is converted to fp16 in shared memory (exact) by warps of their own: with V's codes as they are, a weight would have to be
//       taken apart into terms of eight bits for products of their own (three e4m3 terms for fp16's eleven bits, measured: slower).
//   P'  is rounded to fp16 (half a step of 2^-11, nothing lost above 2^-25 / 2^7 of the reference): M is kept 7 below the
//       largest y and is raised only when a y exceeds it by 15, so p' <= 2^15.  The sum is of the unrounded p', in fp32.
//
// Work.  One CTA per SM walks an even share of the tiles of all (sequence, KV head) units, R rows of them at a time: a
// run may begin and end inside a unit.  Units that one CTA has whole are written at once, the parts of the others go
// to the workspace and join_kernel merges them.  With several row groups CTAs of neighbouring index walk the same tiles
// for different rows, so all but one read them from L2.
//
// Measured (GB300, 32 heads on 8 but for the last, pages of 16 tokens, a scale for 16): 8 single tokens over 1024 to 8192 tokens 27.0 us;
// 4 x 8 nodes over 32768 66 us (4.1 TB/s, 61% of the copy rate: a tile takes some 2000 cycles, of which its shared-memory traffic
// is 1350); 4 x 64 nodes over 32768 140 us and 16 x 60 nodes of 64 heads over 4096 167 us (51% and 40% of the bf16 rate: what
// bounds both is the softmax, 1700 cycles a tile of 128 x 128 scores with the schedulers issuing in 46% of them, then 15000 cycles for a
// unit's beginning and end).
//
// The roles of the warps (struct Cfg) share one instruction cache: code that every tile runs is kept short, and code that runs once per
// unit is rolled up (unrolled, half of the fetches missed and every warp waited for them).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
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
constexpr uint32_t kNoPage = 0x7FDEAD01u;    // in the place of a scale: its key's page has no id
constexpr float kFloor = -INFINITY;          // reference of a row that has met no key
constexpr float kBelow = 7.f, kRise = 15.f;  // the reference lies kBelow under the largest y; raised when exceeded by kRise
// References beyond this make their rows NaN: fp32 holds them to half a unit of the exponent and more, and where rounding passes the
// margins a row would overflow or vanish.
constexpr float kMostM = 4194304.f;
// Rows whose largest |q| * scale reaches this are NaN from the beginning: below it every score lies in fp32's range (at most 2^24
// in Q K, 2^40 of a key's scale and 2^64 of the row's factor), so -inf means that there is no key.
constexpr float kMostQ = 1180591620717411303424.f;  // 2^70
constexpr float kLn2f = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634074f;

// R: queries' rows per CTA.  Up to 32 they are the columns of the products (keys, then channels, in the 128 rows), above they are
// its rows ("wide": R = 128).
template <int R>
struct Cfg {
  static constexpr bool WIDE = R == 128;
  static constexpr int CPT = WIDE ? 64 : 8;                      // scores per softmax thread and tile
  static constexpr int GROUPS = WIDE ? 4 : R / CPT;              // what shares references: a quadrant's two warps, or four warps
  static constexpr int SOFT = WIDE ? 4 * BK / CPT : 4 * GROUPS;
  // Warps: K copies, V and scale copies, K Q^T (and owner of the tensor memory), V^T P^T, converters, softmax.  Up to 32 rows, where a
  // tile should take no longer than its bytes (1400 cycles), two copying warps and two groups of converters take alternate tiles.
  static constexpr int PAIR = WIDE ? 1 : 2;
  static constexpr int W_V = PAIR, W_QK = 2 * PAIR, W_PV = W_QK + 1, W_CONV = W_PV + 1, CONV = 4 * PAIR;
  static constexpr int FIRST_SOFT = W_CONV + CONV;
  static constexpr int THREADS = 32 * (FIRST_SOFT + SOFT);
  static constexpr int SK = 4;
  static constexpr int SV = WIDE ? 3 : 4;
  static constexpr int NP = 2;                                   // P buffers (wide: in tensor memory)
  static constexpr int NV = 2;                                   // fp16 V buffers
  static constexpr uint32_t PROW = 2 * R;                        // bytes of a P^T row, the width of its swizzle
  static constexpr uint32_t QPART = R * HD;                      // one of Q's two parts
  static constexpr uint32_t PBUF = WIDE ? 0 : BK * R * 2;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * QPART;
  static constexpr uint32_t OFF_V = OFF_K + SK * TILE8;
  static constexpr uint32_t OFF_V16 = OFF_V + SV * TILE8;
  static constexpr uint32_t OFF_P = OFF_V16 + NV * TILE16;
  static constexpr uint32_t OFF_RAW = OFF_P + NP * PBUF;         // {ks, vs} per key, kScaleSlots tiles
  // {ks}, {log2 vs}, {1 / vs} of two tiles
  static constexpr uint32_t OFF_SC = OFF_RAW + kScaleSlots * BK * 8;
  static constexpr uint32_t OFF_RM = OFF_SC + 2 * 3 * BK * 4;      // per pair of rows {r0, r1, M0, M1}
  static constexpr uint32_t OFF_R2 = OFF_RM + (WIDE ? 0 : R * 8);  // row scales of the next segment
  static constexpr uint32_t OFF_RED = OFF_R2 + R * 4;            // exchanged maxima and sums
  static constexpr uint32_t OFF_FAC = OFF_RED + 4 * R * 4;
  static constexpr uint32_t OFF_VIS = OFF_FAC + R * 4;           // columns: mask words of the rows
  static constexpr uint32_t OFF_BAR = OFF_VIS + (WIDE ? 0 : R * 32);
  static constexpr int NBAR = 2 * SK + 2 * SV + 2 * NV + 2 + 2 * NP + 2 * kScaleSlots + 2 + 5;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t SMEM = OFF_MISC + 64 + 1024;
  static constexpr uint32_t TMEM_COLS = R == 16 ? 64 : R == 32 ? 128 : 512;
  static constexpr uint32_t COL_S = R;                           // O, then S_0, S_1, wide: P_0, P_1
  static constexpr uint32_t COL_P = 3 * R;
  static_assert(SMEM <= 232448, "shared memory budget");
  // Two copying warps and two groups of converters do not keep each other's order, so each has stages of its own: were they shared, a warp
  // could take the phase before the last for the last and fill a stage that is still to be read.
  static_assert(SK % PAIR == 0 && SV % PAIR == 0 && NV % PAIR == 0 && kScaleSlots % PAIR == 0, "stages of one parity of tiles");
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
  uint32_t q_end;    // (as bits) rows with larger queries are NaN: kMostQ / scale
  float scale_log2;  // scale * log2 e / 4 (the quarter keeps it finite for every finite scale; the rows' factors take it back)
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
// Work is dealt out in tiles' worth of time: a unit takes its tiles and, before them, `begin` for its queries, the pipeline's filling
// and its result.  (By tiles alone the CTAs that begin a unit on their way end last: 58 against 53 us with 4 x 8 nodes over
// 32768 tokens, 132 against 124 with 64 nodes.)  kBegin of 0, 3, 5, 6, 8 and 11: six is best or within 1% of it where CTAs have 50 tiles
// and more (with none chains take 69.2 us for 66.5, 16 x 60 nodes 174 for 170), three with 15 tiles, and where CTAs have few a unit's
// beginning, which each of them has, need not be counted: a quarter of a CTA's tiles at most.
constexpr int kBegin = 6;
struct Time {
  int begin, total;
  __device__ __forceinline__ int of(int T) const { return T > 0 ? T + begin : 0; }
};
__device__ __forceinline__ Time time_of(const Params& p, int lane) {  // (by one warp)
  int N = 0, units = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int T = tiles_of(p, b);
    N += T;
    units += T > 0;
  }
  N = static_cast<int>(__reduce_add_sync(0xffffffffu, N)) * p.Hkv;
  units = static_cast<int>(__reduce_add_sync(0xffffffffu, units)) * p.Hkv;
  Time t;
  t.begin = min(kBegin, N / (4 * p.Gr));
  t.total = N + units * t.begin;
  return t;
}
// The segments of the range [x, x1) of that time, from sequence b on; `off` into its unit h.
struct Walk {
  int x, x1, b, h, off, begin;
  __device__ __forceinline__ bool next(const Params& p, Segment& s) {
    while (x < x1) {
      int T = tiles_of(p, b);
      while (T == 0) {  // (x < x1: a sequence with tiles follows)
        ++b;
        T = tiles_of(p, b);
      }
      const int end = min(T + begin, off + (x1 - x));
      s.b = b, s.h = h, s.T = T, s.L = p.prefix_len[b];
      s.t0 = max(0, off - begin);
      s.t1 = max(0, end - begin);
      x += end - off;
      off = end;
      if (off == T + begin) {
        off = 0;
        if (++h == p.Hkv) h = 0, ++b;
      }
      if (s.t1 > s.t0) return true;
    }
    return false;
  }
};

// How a time of N is dealt out to CTAs: the first `more` of them get one more than `each`.  (No CTA between two parts of a unit is
// without tiles.)
struct Share {
  int each, more;
  __device__ __forceinline__ Share(int N, int Gr) : each(N / Gr), more(N - N / Gr * Gr) {}
  __device__ __forceinline__ int start(int c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int cta_of(int x) const {
    const int wide = more * (each + 1);
    return x < wide ? x / (each + 1) : more + (x - wide) / each;
  }
};

// The run of CTA `cta`: all units of a row group in the order of sequences and heads, dealt out (by one warp).
__device__ __forceinline__ Walk walk_of(const Params& p, const Time& time, int cta, int lane) {
  const Share share(time.total, p.Gr);
  Walk w{share.start(cta), share.start(cta + 1), 0, 0, 0, time.begin};
  int before = 0;
  for (int b0 = 0; b0 < p.B && w.x < w.x1; b0 += 32) {
    const int T = b0 + lane < p.B ? time.of(tiles_of(p, b0 + lane)) : 0;
    int sum = T * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + sum > w.x);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1, Tl = __shfl_sync(0xffffffffu, T, l);
      const int at = w.x - (before + __shfl_sync(0xffffffffu, sum, l) - Tl * p.Hkv);
      w.b = b0 + l;
      w.h = at / Tl;
      w.off = at - w.h * Tl;
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return w;
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
// A from tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, one;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The barrier gets an arrival when the MMAs that the elected lane has issued are done.
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
      "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// Instruction descriptors (fields as in idesc_bf16_f32; format 0 is e4m3 in kind f8f6f4 and fp16 in kind f16, 1 is e5m2).
__host__ __device__ constexpr uint32_t idesc_of(int N, int a_format, int b_format, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_format) << 7) | (static_cast<uint32_t>(b_format) << 10) |
         (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(BK >> 4) << 24);
}
// Four bytes global -> shared, asynchronously, and a lane's arrival once its copies so far have landed.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_copied(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// A key's scales in the exponent's units: y = s a r + lv with the row's factor r, and 1 / vs.
struct KeyScale {
  float a, lv, iv;
};
__device__ __forceinline__ KeyScale key_scale(float2 raw) {
  KeyScale k;
  k.a = scale_in_range(raw.x);
  k.lv = __log2f(scale_in_range(raw.y));
  k.iv = ex2_approx(-k.lv);
  if (__float_as_uint(raw.x) == kNoPage) k = KeyScale{0.f, -INFINITY, 0.f};
  return k;
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
// 16 (or 8) consecutive columns of this thread's lane, and wait for them.
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

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : TS_R8(0)
               : "r"(taddr)
               : "memory");
}
// One column.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(taddr) : "memory");
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}

// Named barriers of the softmax's groups.
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}
__device__ __forceinline__ bool group_any(int group, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + group), "r"(threads), "r"(static_cast<uint32_t>(v))
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
#pragma unroll 1
  do {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  } while (__all_sync(0xffffffffu, *abort_flag == 0 && global_timer_ns() - t0 <= kWaitLimitNs));
  if (*abort_flag == 0) report(status, TS_ERR_TIMEOUT);
  *abort_flag = 1;
  return false;
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

// What the softmax warps need of their CTA.
struct Bars {
  uint32_t s_full, p_full, p_empty, sc_full, q_full, q_empty, o_free;
};
template <int R>
struct Cta {
  const Params& p;
  Bars bar;
  unsigned char* sptr;
  uint32_t tmem;
  volatile int* abort_flag;
  volatile int* nan_seg;
  int rg, cta, R0, rows_here;
  __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const { return wait_warp(b, parity, abort_flag, p.status); }
  // The scores and the scales of buffer s are there.
  __device__ __forceinline__ bool scores_in(int s, uint32_t parity) const {
    const uint32_t a = bar.sc_full + 8 * s, b = bar.s_full + 8 * s;
    if (__all_sync(0xffffffffu, mbar_try(a, parity) && mbar_try(b, parity))) return true;
    return wait(a, parity) && wait(b, parity);
  }
  // P V of tile i is done: its P buffer is free again.  (A barrier of one phase per tile would not do: the softmax may be two tiles
  // ahead of P V, and a wait by parity would take the older phase for the newer.)
  __device__ __forceinline__ bool o_holds(int i) const { return wait(bar.p_empty + 8 * (i & 1), (i >> 1) & 1); }
  __device__ __forceinline__ long long slot(const Segment& s) const {
    return (static_cast<long long>(rg) * p.Gr + cta) * 2 + (s.t0 == 0 ? 1 : 0);
  }
  // index of a row's query, output and log-sum-exp
  __device__ __forceinline__ long long row_at(const Segment& s, int r) const {
    const int row = R0 + r, node = row / p.g;
    return (static_cast<long long>(s.b) * p.m + node) * p.Hq + s.h * p.g + row - node * p.g;
  }
  __device__ __forceinline__ const uint64_t* mask_of(const Segment& s, int r) const {
    return p.mask + (static_cast<long long>(s.b) * p.m + min(R0 + r, p.rows - 1) / p.g) * p.W;
  }
  // V code row of tree node n (nullptr: its page has no id)
  __device__ __forceinline__ const uint8_t* v_row(const Segment& s, int n) const {
    const int pos = s.L + n, id = p.table[static_cast<long long>(s.b) * p.max_blocks + (pos >> p.bs_log2)];
    if (id < 0 || id >= p.num_blocks) return nullptr;
    return p.vc + ((static_cast<long long>(id) * p.Hkv + s.h) * p.bs + (pos & (p.bs - 1))) * HD;
  }
};
__device__ __forceinline__ float lse_of(float M, float l) { return l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2f; }
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Columns are rows: a thread has one key (its TMEM lane) and CPT of the R rows; four warps share the rows' references.
template <int R>
__device__ __forceinline__ void softmax_narrow(const Cta<R>& c, Walk walk, int warp, int lane) {
  using C = Cfg<R>;
  constexpr int N = C::CPT;
  const Params& p = c.p;
  const int quarter = warp & 3, group = (warp - C::FIRST_SOFT) >> 2, col0 = group * N, key = 32 * quarter + lane;
  if (col0 >= c.rows_here) return;  // (what P^T holds in those columns reaches theirs of O^T alone)
  const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16, tO = c.tmem + lanes + col0;
  float* rm = reinterpret_cast<float*>(c.sptr + C::OFF_RM) + 2 * col0;  // {r0, r1, M0, M1} per pair of rows
  float* red = reinterpret_cast<float*>(c.sptr + C::OFF_RED) + col0;    // [quarter * R + row]
  float* factor = reinterpret_cast<float*>(c.sptr + C::OFF_FAC) + col0;
  uint64_t* vis = reinterpret_cast<uint64_t*>(c.sptr + C::OFF_VIS) + 4 * col0;  // mask words of this group's rows
  auto m_at = [&](int r) -> float& { return rm[(r >> 1) * 4 + 2 + (r & 1)]; };
  // P^T [key][row]: rows of PROW bytes, 16-byte chunks swizzled with the key
  const int swz = C::PROW == 64 ? ((key >> 1) & 3) : ((key >> 2) & 1);
  unsigned char* prow = c.sptr + C::OFF_P + key * C::PROW;
  Segment sg;
  bool ok = true;
  int it = 0, seg = 0;
  while (walk.next(p, sg)) {
    if (ok) ok = c.wait(c.bar.q_full, seg & 1);
    if (group_any(group, 128, !ok)) break;
    if (quarter == 0 && lane < N) {
      rm[(lane >> 1) * 4 + (lane & 1)] = reinterpret_cast<const float*>(c.sptr + C::OFF_R2)[col0 + lane];
      m_at(lane) = col0 + lane < c.rows_here ? kFloor : -kFloor;  // (padding: weights 0)
      if (sg.t1 * BK > sg.L) {
        const uint64_t* words = c.mask_of(sg, col0 + lane);
        for (int i = 0; i < p.W; ++i) vis[4 * lane + i] = words[i];
      }
    }
    group_sync(group, 128);
    if (lane == 0) mbar_arrive(c.bar.q_empty);  // (the row scales are taken; the MMA warp says when Q is)
    uint64_t l2[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) l2[i] = 0ull;
    // The rows' constants stay in registers: {r0, r1} and {-M0, -M1}, 0 for the reference of a row that has met no key.
    uint64_t r2[N / 2], m2[N / 2];
    bool unmet = true;
    auto hold = [&]() {
      unmet = false;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float4 k = reinterpret_cast<const float4*>(rm)[i];
        r2[i] = pack_f32x2(k.x, k.y);
        m2[i] = pack_f32x2(k.z == kFloor ? 0.f : -k.z, k.w == kFloor ? 0.f : -k.w);
        unmet = unmet || k.z == kFloor || k.w == kFloor;
      }
    };
    hold();
    bool left = false;
    for (int t = sg.t0; t < sg.t1; ++t, ++it) {
      const int s = it & 1;
      const bool tail = (t + 1) * BK > sg.L;
      const uint32_t tS = c.tmem + lanes + C::COL_S + R * s + col0;
      if (ok) ok = c.scores_in(s, (it >> 1) & 1);
      KeyScale k = {0.f, 0.f, 0.f};
      uint32_t x[N];
      uint32_t seen = ~0u;  // rows that attend to this thread's key
      if (ok) {
        tc_fence_after();
        const float* sc = reinterpret_cast<const float*>(c.sptr + C::OFF_SC) + s * 3 * BK + key;
        k = KeyScale{sc[0], sc[BK], sc[2 * BK]};
        if (tail) {
          const int n = t * BK + key - sg.L;
          if (k.iv == 0.f || n >= p.m) {
            seen = 0u;
          } else if (n >= 0) {
            seen = 0u;
#pragma unroll 4
            for (int i = 0; i < N; ++i) seen |= static_cast<uint32_t>((vis[i * 4 + (n >> 6)] >> (n & 63)) & 1ull) << i;
          }
        }
      }
      const uint64_t a2 = pack_f32x2(k.a, k.a), v2 = pack_f32x2(k.lv, k.lv);
#pragma unroll 1
      for (bool again = false;; again = true) {
        float top = -INFINITY, top2 = -INFINITY;
        if (ok) {
          tmem_ld(tS, x);
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const uint64_t z2 = fma_f32x2(pack_f32x2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), mul_f32x2(a2, r2[i / 2]),
                                          add_f32x2(v2, m2[i / 2]));
            float z0, z1;
            unpack_f32x2(z2, z0, z1);
            x[i] = __float_as_uint(z0);
            x[i + 1] = __float_as_uint(z1);
          }
          if (tail) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (!((seen >> i) & 1u)) x[i] = 0xFF800000u;
          }
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            top = max3(top, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            top2 = max3(top2, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
          top = fmaxf(top, top2);
        }
        if (again || !group_any(group, 128, !ok || unmet || top > kRise)) break;
        // Rare (every unit's first tile does this): the references rise to the tile's largest, and the scores are taken again.
        if (group_any(group, 128, !ok)) {
          left = true;
          break;
        }
        int high = 0x80000000;
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          float y = fmaf(tmem_ld1(tS + i), k.a * rm[(i >> 1) * 4 + (i & 1)], k.lv);
          if (y != y || !((seen >> i) & 1u)) y = -INFINITY;  // (a NaN goes into the weights, not into the reference)
          const int most = __reduce_max_sync(0xffffffffu, ordered(y));
          if (lane == i) high = most;
        }
        if (lane < N) red[quarter * R + lane] = from_ordered(high);
        group_sync(group, 128);
        if (quarter == 0 && lane < N) {
          const float old = m_at(lane);
          const float M = fmaxf(fmaxf(red[lane], red[R + lane]), fmaxf(red[2 * R + lane], red[3 * R + lane])) - kBelow;
          const bool rises = M > old;  // (kFloor before the first key, and nothing where there is none yet)
          factor[lane] = rises && old != kFloor ? ex2_approx(old - M) : 1.f;
          if (rises) m_at(lane) = fabsf(M) > kMostM ? __int_as_float(0x7FC00000) : M;
        }
        group_sync(group, 128);
        hold();
#pragma unroll
        for (int i = 0; i < N / 2; ++i) l2[i] = mul_f32x2(l2[i], *reinterpret_cast<const uint64_t*>(factor + 2 * i));
        if (t > sg.t0) {
          ok = c.o_holds(it - 1);
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < N; ++i) tmem_st1(tO + i, tmem_ld1(tO + i) * factor[i]);
            tmem_st_wait();
          }
        }
      }
      if (left) break;
      if (!ok) continue;  // (leaves at the next vote)
      const uint64_t iv2 = pack_f32x2(k.iv, k.iv);
      uint32_t h[N / 2];
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float p0 = ex2_approx(__uint_as_float(x[i])), p1 = ex2_approx(__uint_as_float(x[i + 1]));
        l2[i / 2] = fma_f32x2(pack_f32x2(p0, p1), iv2, l2[i / 2]);
        h[i / 2] = pack_f16x2(p0, p1);
      }
#pragma unroll
      for (int j = 0; j < N / 8; ++j)
        *reinterpret_cast<uint4*>(prow + s * C::PBUF + (((col0 / 8 + j) ^ swz) << 4)) =
            make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar.p_full + 8 * s);
    }
    if (left) ok = false;
    if (ok) ok = c.o_holds(it - 1);
    if (group_any(group, 128, !ok)) break;
    // ------------------------------ the segment's result ------------------------------
    tc_fence_after();
    float lv[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) unpack_f32x2(l2[i], lv[2 * i], lv[2 * i + 1]);
    const float mine = column_sums(lv, lane);  // lane i: column i's sum over this warp's keys
    if (lane < N) red[quarter * R + lane] = mine;
    group_sync(group, 128);
    const bool whole = sg.t0 == 0 && sg.t1 == sg.T;
    const long long slot_at = c.slot(sg) * R + col0;
    float l = 0.f;
    if (lane < N) {
      l = (red[lane] + red[R + lane]) + (red[2 * R + lane] + red[3 * R + lane]);
      if (quarter == 0 && col0 + lane < c.rows_here) {
        if (!whole) p.part_ml[slot_at + lane] = make_float2(m_at(lane), l);
        else if (p.lse != nullptr) p.lse[c.row_at(sg, col0 + lane)] = lse_of(m_at(lane), l);
      }
    }
    const float inv = whole ? inverse(l) : 1.f;
    const bool poison = c.nan_seg[seg & 1] == seg + 1;
#pragma unroll 1
    for (int i = 0; i < min(N, c.rows_here - col0); ++i) {
      float o = tmem_ld1(tO + i) * __shfl_sync(0xffffffffu, inv, i);
      if (poison) {
        // a NaN in a tree row's V: the rows that attend to it get it (this thread has channel `key`)
        for (int n = max(0, sg.t0 * BK - sg.L); n < min(p.m, sg.t1 * BK - sg.L); ++n) {
          const uint8_t* v = c.v_row(sg, n);
          if (v != nullptr && (v[key] & 0x7Fu) == 0x7Fu && ((vis[4 * i + (n >> 6)] >> (n & 63)) & 1ull)) o = __int_as_float(0x7FC00000);
        }
      }
      if (whole) p.out[c.row_at(sg, col0 + i) * HD + key] = __float2bfloat16_rn(o);
      else p.part_o[(slot_at + i) * HD + key] = o;
      __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar.o_free);
    group_sync(group, 128);  // (red and the references are written again)
    ++seg;
  }
}

// Keys kb .. kb + 63 that a row attends to: the prefix, then the bits of its mask words for the tree, nothing behind it.
__device__ __forceinline__ uint64_t visible64(int kb, int L, int m, const uint64_t* words, int W) {
  const int pre = L - kb;
  if (pre >= 64) return ~0ull;
  const int n0 = max(0, -pre);  // first tree node among the keys
  uint64_t bits = 0ull;
  if (n0 < m) {
    const int q = n0 >> 6, sh = n0 & 63;
    bits = words[q] >> sh;
    if (sh != 0 && q + 1 < W) bits |= words[q + 1] << (64 - sh);
    if (m - n0 < 64) bits &= (1ull << (m - n0)) - 1ull;
  }
  return pre > 0 ? ((1ull << pre) - 1ull) | (bits << pre) : bits;
}

// Rows are rows: a thread has one row (its TMEM lane) and N of the tile's keys, the thread of the warp four further on the
// others; both keep the row's reference.  P goes to tensor memory.
// GROUP keys have one scale (16, 4 or 1, as the scale blocks allow): it is folded into the row's constants once for as many scores.
// With a scale for each key, reading them (a broadcast of 16 bytes to a warp takes the shared memory four cycles) is what paces the
// softmax: 4 x 64 nodes of 32 heads over 32768 tokens take 141 us with a scale for 16, 152 with one for 4 or 8 (172 by keys), 170 with
// one for each.
template <int R, int GROUP>
__device__ __forceinline__ void softmax_wide(const Cta<R>& c, Walk walk, int warp, int lane) {
  using C = Cfg<R>;
  constexpr int N = C::CPT, PARTS = BK / N;
  const Params& p = c.p;
  const int quad = warp & 3, part = (warp - C::FIRST_SOFT) >> 2, row = 32 * quad + lane;
  if (32 * quad >= c.rows_here) return;
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16, tO = c.tmem + lanes + N * part;
  float* red = reinterpret_cast<float*>(c.sptr + C::OFF_RED);  // [part][row]
  const bool valid = row < c.rows_here;
  Segment sg;
  bool ok = true;
  int it = 0, seg = 0;
  while (walk.next(p, sg)) {
    if (ok) ok = c.wait(c.bar.q_full, seg & 1);
    if (group_any(quad, 32 * PARTS, !ok)) break;
    const float r = reinterpret_cast<const float*>(c.sptr + C::OFF_R2)[row];
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar.q_empty);  // (the row scale is taken; the MMA warp says when Q is)
    const uint64_t* words = c.mask_of(sg, row);
    float M = valid ? kFloor : -kFloor;  // (padding: weights 0)
    uint64_t l2 = 0ull;
    bool left = false;
    for (int t = sg.t0; t < sg.t1; ++t, ++it) {
      const int s = it & 1;
      if (ok) ok = c.scores_in(s, (it >> 1) & 1);
      const float* sc = reinterpret_cast<const float*>(c.sptr + C::OFF_SC) + s * 3 * BK + N * part;  // a, lv, iv of this part's keys
      uint32_t x[N];
      const bool tail = (t + 1) * BK > sg.L;
      if (ok) tc_fence_after();
#pragma unroll 1
      for (bool again = false;; again = true) {
        float top = -INFINITY, top2 = -INFINITY;
        if (ok) {
          tmem_ld64(c.tmem + lanes + C::COL_S + BK * s + N * part, x);
          const float ref = M == kFloor ? 0.f : -M;
          if constexpr (GROUP > 1) {
#pragma unroll
            for (int g = 0; g < N; g += GROUP) {
              const float a = sc[g] * r, b = sc[BK + g] + ref;
              const uint64_t a2 = pack_f32x2(a, a), b2 = pack_f32x2(b, b);
#pragma unroll
              for (int i = g; i < g + GROUP; i += 2) {
                float z0, z1;
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), a2, b2), z0, z1);
                x[i] = __float_as_uint(z0);
                x[i + 1] = __float_as_uint(z1);
              }
            }
          } else {
            const uint64_t r2 = pack_f32x2(r, r), m2 = pack_f32x2(ref, ref);
#pragma unroll
            for (int i = 0; i < N; i += 4) {
              const float4 a = *reinterpret_cast<const float4*>(sc + i), v = *reinterpret_cast<const float4*>(sc + BK + i);
              const uint64_t z01 = fma_f32x2(pack_f32x2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                             mul_f32x2(pack_f32x2(a.x, a.y), r2), add_f32x2(pack_f32x2(v.x, v.y), m2));
              const uint64_t z23 = fma_f32x2(pack_f32x2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])),
                                             mul_f32x2(pack_f32x2(a.z, a.w), r2), add_f32x2(pack_f32x2(v.z, v.w), m2));
              float z[4];
              unpack_f32x2(z01, z[0], z[1]);
              unpack_f32x2(z23, z[2], z[3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) x[i + j] = __float_as_uint(z[j]);
            }
          }
          if (tail) {
            const uint64_t vis = (visible64(t * BK + N * part, sg.L, p.m, words, p.W));
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (!((vis >> i) & 1ull) || sc[2 * BK + i] == 0.f) x[i] = 0xFF800000u;
          }
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            top = max3(top, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            top2 = max3(top2, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
          top = fmaxf(top, top2);
        }
        if (again || !group_any(quad, 32 * PARTS, !ok || top > kRise || (M == kFloor && top > -INFINITY))) break;
        // Rare (every unit's first tile does this): the reference rises to the tile's largest, and the scores are taken again.
        if (group_any(quad, 32 * PARTS, !ok)) {
          left = true;
          break;
        }
        red[part * R + row] = top;
        group_sync(quad, 32 * PARTS);
        float most = red[row];
#pragma unroll
        for (int i = 1; i < PARTS; ++i) most = fmaxf(most, red[i * R + row]);
        const float high = (M == kFloor ? 0.f : M) + most - kBelow;
        group_sync(quad, 32 * PARTS);  // (red is written again)
        const bool rises = high > M;
        const float f = rises && M != kFloor ? ex2_approx(M - high) : 1.f;
        if (rises) M = fabsf(high) > kMostM && valid ? __int_as_float(0x7FC00000) : high;
        l2 = mul_f32x2(l2, pack_f32x2(f, f));
        if (t > sg.t0) {
          ok = c.o_holds(it - 1);
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < N; i += 16) {
              uint32_t o[16];
              tmem_ld(tO + i, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st(tO + i, o);
            }
            tmem_st_wait();
          }
        }
      }
      if (left) break;
      if (!ok) continue;  // (leaves at the next vote)
#pragma unroll
      for (int i = 0; i < N; i += 32) {
        uint32_t h[16];
        uint64_t sum = 0ull;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float p0 = ex2_approx(__uint_as_float(x[i + j])), p1 = ex2_approx(__uint_as_float(x[i + j + 1]));
          const float p2 = ex2_approx(__uint_as_float(x[i + j + 2])), p3 = ex2_approx(__uint_as_float(x[i + j + 3]));
          if constexpr (GROUP > 1) {
            sum = add_f32x2(sum, add_f32x2(pack_f32x2(p0, p1), pack_f32x2(p2, p3)));
            if (j % GROUP == GROUP - 4) {
              const float iv = sc[2 * BK + i + j + 4 - GROUP];
              l2 = fma_f32x2(sum, pack_f32x2(iv, iv), l2);
              sum = 0ull;
            }
          } else {
            const float4 v = *reinterpret_cast<const float4*>(sc + 2 * BK + i + j);
            l2 = fma_f32x2(pack_f32x2(p0, p1), pack_f32x2(v.x, v.y), l2);
            l2 = fma_f32x2(pack_f32x2(p2, p3), pack_f32x2(v.z, v.w), l2);
          }
          h[j / 2] = pack_f16x2(p0, p1);
          h[j / 2 + 1] = pack_f16x2(p2, p3);
        }
        tmem_st(c.tmem + lanes + C::COL_P + 64 * s + N / 2 * part + i / 2, h);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar.p_full + 8 * s);
    }
    if (left) ok = false;
    if (ok) ok = c.o_holds(it - 1);
    if (group_any(quad, 32 * PARTS, !ok)) break;
    // ------------------------------ the segment's result ------------------------------
    tc_fence_after();
    float l, other;
    unpack_f32x2(l2, l, other);
    l += other;
    red[part * R + row] = l;
    group_sync(quad, 32 * PARTS);
    l = red[row];  // (all threads in the same order)
#pragma unroll
    for (int i = 1; i < PARTS; ++i) l += red[i * R + row];
    const bool whole = sg.t0 == 0 && sg.t1 == sg.T, poison = c.nan_seg[seg & 1] == seg + 1;
    const long long to = whole ? c.row_at(sg, row) : c.slot(sg) * R + row;
    if (valid && part == 0) {
      if (!whole) p.part_ml[to] = make_float2(M, l);
      else if (p.lse != nullptr) p.lse[to] = lse_of(M, l);
    }
    const float inv = whole ? inverse(l) : 1.f;
#pragma unroll 1
    for (int i = 0; i < N; i += 16) {
      uint32_t o[16];
      tmem_ld(tO + i, o);
      const int ch = N * part + i;
      if (poison) {
        // a NaN in a tree row's V: the rows that attend to it get it
        for (int n = max(0, sg.t0 * BK - sg.L); n < min(p.m, sg.t1 * BK - sg.L); ++n) {
          const uint8_t* v = c.v_row(sg, n);
          if (v == nullptr || !((words[n >> 6] >> (n & 63)) & 1ull)) continue;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((v[ch + j] & 0x7Fu) == 0x7Fu) o[j] = 0x7FC00000u;
        }
      }
      float f[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(o[j]) * inv;
      if (whole && valid) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + to * HD + ch);
        dst[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        dst[1] = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]), pack_bf16x2(f[12], f[13]), pack_bf16x2(f[14], f[15]));
      } else if (valid) {
        float4* dst = reinterpret_cast<float4*>(p.part_o + to * HD + ch);
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar.o_free);
    group_sync(quad, 32 * PARTS);  // (red is written again)
    ++seg;
  }
}

__device__ const uint32_t g_no_page[1] = {kNoPage};

// Block ids of a segment's pages by one warp: a lane holds one of 32, the next 32 are on their way.
struct Pages {
  int now, next, base, end, first;  // base: index (in the segment) of `now`'s first
  __device__ __forceinline__ void begin(const Params& p, const Segment& s, int ppt, int lane) {
    first = s.t0 * ppt;
    end = (s.L + p.m + p.bs - 1) >> p.bs_log2;
    base = 0;
    now = block_at(p, s.b, first + lane, end);
    next = block_at(p, s.b, first + 32 + lane, end);
  }
  // Makes `now` hold pages i .. (tile by tile; a tile's pages never straddle: both are powers of two).
  __device__ __forceinline__ void seek(const Params& p, const Segment& s, int i, int lane) {
    if (i < base + 32) return;
    base += 32;
    now = next;
    next = block_at(p, s.b, first + base + 32 + lane, end);
  }
};

template <int R, int GROUP>
__global__ void __launch_bounds__(Cfg<R>::THREADS, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const __grid_constant__ Params p) {
  using C = Cfg<R>;
  constexpr int SK = C::SK, SV = C::SV, NP = C::NP, NV = C::NV;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* sptr = smem_raw + (sbase - raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rg = blockIdx.x % p.RG, cta = blockIdx.x / p.RG;
  const int R0 = rg * R, rows_here = min(R, p.rows - R0);
  // softmax warps whose rows (wide: quadrants of 32, otherwise columns of CPT) hold any; the others have nothing to do
  const int soft = C::WIDE ? BK / C::CPT * ((rows_here + 31) / 32) : 4 * ((rows_here + C::CPT - 1) / C::CPT);

  uint32_t at = sbase + C::OFF_BAR;
  auto take = [&](int n) {
    const uint32_t first = at;
    at += 8u * n;
    return first;
  };
  const uint32_t full_k = take(SK), empty_k = take(SK), full_v = take(SV), empty_v = take(SV), v16_full = take(NV),
                 v16_empty = take(NV), s_full = take(2), p_full = take(NP), p_empty = take(NP),
                 raw_full = take(kScaleSlots), raw_empty = take(kScaleSlots), sc_full = take(2),
                 q_full = take(1), q_empty = take(1), o_free = take(1), last = take(2);
  unsigned char* misc = sptr + C::OFF_MISC;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* nan_seg = reinterpret_cast<volatile int*>(misc + 8);  // [2]: the segment (+1) whose tree rows have NaN in V
  Walk* s_walk = reinterpret_cast<Walk*>(misc + 16);

  if (threadIdx.x == 0) {
    for (int i = 0; i < SK; ++i) mbar_init(full_k + 8 * i, 1), mbar_init(empty_k + 8 * i, 1);
    for (int i = 0; i < SV; ++i) mbar_init(full_v + 8 * i, 1), mbar_init(empty_v + 8 * i, 4);
    for (int i = 0; i < NV; ++i) mbar_init(v16_full + 8 * i, 4), mbar_init(v16_empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(s_full + 8 * i, 1), mbar_init(sc_full + 8 * i, 4);
    for (int i = 0; i < NP; ++i) mbar_init(p_full + 8 * i, soft), mbar_init(p_empty + 8 * i, 1);
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(raw_full + 8 * i, 32), mbar_init(raw_empty + 8 * i, 4);
    mbar_init(q_full, C::CONV);
    mbar_init(q_empty, 1 + soft);
    mbar_init(o_free, soft);
    mbar_init(last, 1);
    mbar_init(last + 8, 1);
    *abort_flag = 0;
    nan_seg[0] = nan_seg[1] = 0;
    fence_mbar_init();
  }
  if (warp == C::W_QK) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 0) {
    const Walk w = walk_of(p, time_of(p, lane), cta, lane);
    if (lane == 0) *s_walk = w;
    if (blockIdx.x == 0)
      for (int b = lane; b < p.B; b += 32)
        if (tiles_of(p, b) == 0) report(p.status, TS_ERR_DEVICE_CHECK);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
  Walk walk = *s_walk;
  Segment sg;
  const int ppt = BK >> p.bs_log2;  // pages per tile
  bool ok = true;

  if (warp < C::W_QK) {
    // ------------------------------ codes by TMA (K, V); V's warps also copy the scales, as they are ------------------------------
    const bool is_k = warp < C::W_V;
    const int part = warp % C::PAIR;
    const int stages = is_k ? SK : SV;
    const uint32_t full = is_k ? full_k : full_v, empty = is_k ? empty_k : empty_v;
    const uint32_t ring = sbase + (is_k ? C::OFF_K : C::OFF_V), box = p.bs * HD;
    const CUtensorMap* map = is_k ? &tmk : &tmv;
    int before = 0, issued = 0;  // tiles of earlier segments; tiles whose copies were issued, by this warp's count
    Pages pg;
    while (ok && walk.next(p, sg)) {
      pg.begin(p, sg, ppt, lane);
      const int n = sg.t1 - sg.t0;
#pragma unroll 1
      for (int t = (before + part) % C::PAIR; t < n; t += C::PAIR) {
        const int i = t * ppt, it = before + t;
        pg.seek(p, sg, i, lane);
        if (!is_k) {
          const int slot = it % kScaleSlots;
          if (pg.now == -1) report(p.status, TS_ERR_DEVICE_CHECK);
          ok = wait_warp(raw_empty + 8 * slot, ((it / kScaleSlots) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = 32 * j + lane;
            const int id = __shfl_sync(0xffffffffu, pg.now, i - pg.base + (key >> p.bs_log2));
            const long long o = (static_cast<long long>(id) * p.Hkv + sg.h) * p.nsb + ((key & (p.bs - 1)) >> p.sb_log2);
            const float* none = reinterpret_cast<const float*>(g_no_page);
            const uint32_t to = sbase + C::OFF_RAW + (slot * BK + key) * 8;
            copy4(to, id >= 0 ? p.ks + o : none);
            copy4(to + 4, id >= 0 ? p.vs + o : none);
          }
          arrive_copied(raw_full + 8 * slot);
        }
        const int round = is_k ? it / SK : it / SV, stage = it - round * stages;
        ok = wait_warp(empty + 8 * stage, (round & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full + 8 * stage, TILE8);
        __syncwarp();
        const uint32_t to = ring + stage * TILE8;
        const int id = __shfl_sync(0xffffffffu, pg.now, i - pg.base + lane);
        if (lane < ppt) tma_load_4d(to + lane * box, map, full + 8 * stage, 0, 0, sg.h, id < 0 ? p.num_blocks : id);
        __syncwarp();
        issued = it + 1;
      }
      before += n;
    }
    // after an abort nobody waits for what is still on its way: this warp's newest copy of every stage
    if (!ok)
      for (int i = max(0, issued - stages * C::PAIR); i < issued; ++i)
        if (i % C::PAIR == part) drain(full + 8 * (i % stages), (i / stages) & 1);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == C::W_QK) {
    // ------------------------------ scores: K Q^T, wide Q K^T (the warp issues as one) ------------------------------
    constexpr int N = C::WIDE ? BK : R;
    constexpr uint32_t iq1 = idesc_of(N, 0, 0, 0, 0), iq2 = C::WIDE ? idesc_of(N, 1, 0, 0, 0) : idesc_of(N, 0, 1, 0, 0);
    const uint64_t kdesc = sdesc(sbase + C::OFF_K, 16, 1024, 128), qdesc = sdesc(sbase + C::OFF_Q, 16, 1024, 128);
    int it = 0, seg = 0, sk = 0, phase = 0;
    while (ok && walk.next(p, sg)) {
      ok = wait_warp(q_full, seg & 1, abort_flag, p.status);
      if (!ok) break;
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int s = it & 1;
        // (P V of the tile before last is done: then its weights have been made, so its scores have been read, and the softmax need
        // not wait for its P buffer)
        ok = wait_warp(full_k + 8 * sk, phase, abort_flag, p.status) &&
             wait_warp(p_empty + 8 * s, ((it >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + C::COL_S + N * s;
        // (descriptors count 16-byte units: a step of 32 bytes adds 2)
        const uint64_t kd = kdesc + static_cast<uint64_t>(sk * (TILE8 >> 4));
#pragma unroll
        for (int kk = 0; kk < 2 * HD / 32; ++kk) {
          const uint64_t a = kd + 2u * (kk & 3), b = qdesc + (C::QPART >> 4) * (kk >> 2) + 2u * (kk & 3);
          if (C::WIDE) mma_f8(d, b, a, kk < 4 ? iq1 : iq2, kk > 0 ? 1u : 0u);
          else mma_f8(d, a, b, kk < 4 ? iq1 : iq2, kk > 0 ? 1u : 0u);
        }
        commit_elected(s_full + 8 * s);
        commit_elected(empty_k + 8 * sk);
        if (++sk == SK) sk = 0, phase ^= 1;
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
  } else if (warp == C::W_PV) {
    // ------------------------------ outputs: V^T P^T, wide P V ------------------------------
    constexpr uint32_t ip = C::WIDE ? idesc_of(HD, 0, 0, 0, 1) : idesc_of(R, 0, 0, 1, 1);
    const uint64_t vdesc = sdesc(sbase + C::OFF_V16, BK * 128, 1024, 128);
    const uint64_t pdesc = sdesc(sbase + C::OFF_P, BK * 128, 8 * C::PROW, C::PROW);
    int it = 0, seg = 0;
    while (ok && walk.next(p, sg)) {
      // (the accumulator is free once the last segment's has been read)
      ok = wait_warp(o_free, (seg & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        const int b = it & 1, phase = (it >> 1) & 1;
        ok = wait_warp(v16_full + 8 * b, phase, abort_flag, p.status) && wait_warp(p_full + 8 * b, phase, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vdesc + static_cast<uint64_t>(b * (TILE16 >> 4)), pd = pdesc + static_cast<uint64_t>(b * (C::PBUF >> 4));
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint32_t more = kk > 0 || t > sg.t0 ? 1u : 0u;
          if (C::WIDE) mma_f16_ts(tmem, tmem + C::COL_P + 64 * b + 8 * kk, vd + (2048u >> 4) * kk, ip, more);
          else mma_f16(tmem, vd + (2048u >> 4) * kk, pd + C::PROW * kk, ip, more);
        }
        commit_elected(v16_empty + 8 * b);
        commit_elected(p_empty + 8 * b);
      }
      ++seg;
    }
    if (!ok) {
      commit_elected(last + 8);
      drain(last + 8, 0);
    }
  } else if (warp < C::FIRST_SOFT) {
    // ------------------------------ Q and V into the tensor cores' types ------------------------------
    const int cw = warp - C::W_CONV, w = cw & 3, part = cw >> 2;  // (w: keys 32 w .. of every tile of this group)
    int before = 0, seg = 0;
    while (ok && walk.next(p, sg)) {
      // eight lanes per row, 16 values each; all rows are asked for before the wait and the first of them
      auto q_at = [&](int r) {
        const int row = R0 + r, node = row / p.g;
        return p.q + ((static_cast<long long>(sg.b) * p.m + node) * p.Hq + sg.h * p.g + row - node * p.g) * HD;
      };
      for (int r = 4 * cw + (lane >> 3); r < rows_here; r += 4 * C::CONV)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(q_at(r) + 16 * (lane & 7)));
      ok = wait_warp(q_empty, (seg & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
#pragma unroll 1
      for (int r0 = cw * 4; r0 < R; r0 += 4 * C::CONV) {
        const int r = r0 + (lane >> 3), c = lane & 7;
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (r < rows_here) {
          const uint4* src = reinterpret_cast<const uint4*>(q_at(r)) + 2 * c;
          x[0] = __ldg(src);
          x[1] = __ldg(src + 1);
        }
        const uint32_t in[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
        uint32_t big = 0;  // largest magnitude, as bits (from q_end on, infinities and NaN among it, the row becomes NaN)
#pragma unroll
        for (int j = 0; j < 8; ++j) big = max(big, max((in[j] << 16) & 0x7FFF0000u, in[j] & 0x7FFF0000u));
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
            const float y0 = bf16_lo(in[2 * j + u]) * f0 * f1, y1 = bf16_hi(in[2 * j + u]) * f0 * f1;
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
        // The row's factor, 2^e * scale * log2 e.  (Not 2^e alone, with the rest in the keys': below 2^-126 there is no such float, and a
        // large scale makes ordinary scores of such rows.)
        const float factor = pow2(e / 2) * p.scale_log2 * pow2(e - e / 2 + 2);
        if (c == 0) reinterpret_cast<float*>(sptr + C::OFF_R2)[r] = big >= p.q_end ? __int_as_float(0x7FC00000) : factor;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      const int n = sg.t1 - sg.t0;
#pragma unroll 1
      for (int i = (before + part) % C::PAIR; i < n; i += C::PAIR) {
        const int t = sg.t0 + i, it = before + i, v = it & 1, sv = it % SV, phase = (it / SV) & 1;
        {
          // the tile's scales as the softmax wants them: a key per thread (P V of the tile before last is done, so they have been read)
          const int slot = it % kScaleSlots, key = 32 * w + lane;
          ok = wait_warp(raw_full + 8 * slot, (it / kScaleSlots) & 1, abort_flag, p.status) &&
               wait_warp(v16_empty + 8 * v, ((it >> 1) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          const KeyScale k = key_scale(reinterpret_cast<const float2*>(sptr + C::OFF_RAW)[slot * BK + key]);
          float* to = reinterpret_cast<float*>(sptr + C::OFF_SC) + v * 3 * BK;
          to[key] = k.a;
          to[BK + key] = k.lv;
          to[2 * BK + key] = k.iv;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(raw_empty + 8 * slot);
            mbar_arrive(sc_full + 8 * v);
          }
        }
        ok = wait_warp(full_v + 8 * sv, phase, abort_flag, p.status);
        if (!ok) break;
        const unsigned char* from = sptr + C::OFF_V + sv * TILE8;
        unsigned char* to = sptr + C::OFF_V16 + v * TILE16;
        // Keys in groups of eight; of a group, lanes of one eighth of the warp take keys k and k ^ 5 and four 16-byte chunks:
        // reads (chunk c at c ^ (k % 8)) and writes (chunks 2c, 2c + 1 of the half's 128-byte row, the same way) then touch
        // all banks once.
        const int pair = lane >> 3, k8 = (lane & 4) ? pair ^ 5 : pair, c4 = lane & 3, k0 = 32 * w + k8;
        // (all loads first: with a branch and a store between them each waited for its own, 2400 cycles a tile)
        uint4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          x[u] = *reinterpret_cast<const uint4*>(from + (k0 + 8 * (u >> 1)) * 128 + (((c4 + 4 * (u & 1)) ^ k8) << 4));
        if ((t + 1) * BK > sg.L) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int pos = t * BK + k0 + 8 * (u >> 1);
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
          unsigned char* row = to + (u & 1) * (BK * 128) + (k0 + 8 * (u >> 1)) * 128;
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
      before += n;
      ++seg;
    }
  } else {
    const Bars bars{s_full, p_full, p_empty, sc_full, q_full, q_empty, o_free};
    const Cta<R> c{p, bars, sptr, tmem, abort_flag, nan_seg, rg, cta, R0, rows_here};
    if constexpr (C::WIDE) softmax_wide<R, GROUP>(c, walk, warp, lane);
    else softmax_narrow(c, walk, warp, lane);
  }
  __syncthreads();
  if (warp == C::W_QK) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Joins the parts of the units that several CTAs walked, in the order of the CTAs, a warp per row.  Either the warps are those of all
// rows of the output, and a row whose unit one CTA had is passed over, or (BOUNDARIES) those of the rows at every boundary between
// two of attn_kernel's CTAs, of which the first inside a unit has the unit.  The form with fewer warps is taken: with 61440 rows
// (16 x 60 nodes of 64 heads) the call takes 173 us by boundaries against 186 by rows, with 1024 (4 x 8 nodes of 32) 68 by
// rows against 71.
constexpr int kJoinWarps = 8, kJoinRows = 32;  // rows of a CTA at a boundary
template <int R, bool BOUNDARIES>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Time time = time_of(p, lane);
  int b, h, rg, r, r1, first;  // unit, row group, rows r, r + kJoinWarps, .. below r1 of it; the place of its first tile
  if constexpr (BOUNDARIES) {
    rg = blockIdx.x % p.RG;
    // (every warp finds the place by itself: no barrier)
    const Walk w = walk_of(p, time, blockIdx.x / p.RG + 1, lane);
    if (w.x >= w.x1 || w.off <= time.begin) return;  // nothing from here on, or a unit begins here
    b = w.b, h = w.h, first = w.x - w.off + time.begin;
    r = blockIdx.y * kJoinRows + warp;
    r1 = min(min(R, p.rows - rg * R), static_cast<int>(blockIdx.y + 1) * kJoinRows);
  } else {
    const long long item = static_cast<long long>(blockIdx.x) * kJoinWarps + warp;
    if (item >= static_cast<long long>(p.B) * p.Hkv * p.rows) return;
    const int bh = static_cast<int>(item / p.rows), row = static_cast<int>(item - static_cast<long long>(bh) * p.rows);
    b = bh / p.Hkv, h = bh - b * p.Hkv, rg = row / R, r = row - rg * R, r1 = r + 1, first = 0;
  }
  const int T = tiles_of(p, b);
  if (T == 0) return;
  if constexpr (!BOUNDARIES) {
    int before = 0;  // time of the sequences before b
    for (int i = lane; i < b; i += 32) before += time.of(tiles_of(p, i));
    first = static_cast<int>(__reduce_add_sync(0xffffffffu, before)) * p.Hkv + h * (T + time.begin) + time.begin;
  }
  const Share share(time.total, p.Gr);
  const int c0 = share.cta_of(first), last = share.cta_of(first + T - 1);
  // one CTA had the whole unit, or an earlier boundary has it
  if (BOUNDARIES ? c0 + 1 != static_cast<int>(blockIdx.x) / p.RG + 1 : c0 == last) return;
  auto slot = [&](int c) { return (static_cast<long long>(rg) * p.Gr + c) * 2 + (c == c0 ? 1 : 0); };
  for (; r < r1; r += kJoinWarps) {
    // (the first parts are asked for together with the references)
    auto part = [&](int c) { return *reinterpret_cast<const float4*>(p.part_o + (slot(c) * R + r) * HD + 4 * lane); };
    constexpr int AHEAD = 4;
    float4 o[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) o[i] = part(min(c0 + i, last));
    float M = -INFINITY;
    for (int c = c0 + lane; c <= last; c += 32) M = fmaxf(M, p.part_ml[slot(c) * R + r].x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int c, const float4& x) {
      const float2 ml = p.part_ml[slot(c) * R + r];
      const float f = ml.x == M ? 1.f : ex2_approx(ml.x - M);
      l = fmaf(ml.y, f, l);
      acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y), acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (c0 + i <= last) add(c0 + i, o[i]);
#pragma unroll 4
    for (int c = c0 + AHEAD; c <= last; ++c) add(c, part(c));
    const int row = rg * R + r, node = row / p.g, head = h * p.g + row % p.g;
    const long long at = (static_cast<long long>(b) * p.m + node) * p.Hq + head;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p.out + at * HD + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse != nullptr) p.lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2f;
  }
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
  pl.R = rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
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

template <int R, int GROUP>
int launch(const Params& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attn_kernel<R, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<R>::SMEM);
  });
  if (e != cudaSuccess) return TS_ERR_CUDA;
  e = launch_pdl(attn_kernel<R, GROUP>, dim3(p.RG * p.Gr), dim3(Cfg<R>::THREADS), Cfg<R>::SMEM, stream, mk, mv, p);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  int launches = 1;
  if (p.Gr > 1) {
    const long long rows = static_cast<long long>(p.B) * p.Hkv * p.rows, blocks = (rows + kJoinWarps - 1) / kJoinWarps;
    const dim3 by(p.RG * (p.Gr - 1), (std::min(R, p.rows) + kJoinRows - 1) / kJoinRows);
    e = blocks <= static_cast<long long>(by.x) * by.y * (kJoinRows / kJoinWarps)
            ? launch_pdl(join_kernel<R, false>, dim3(static_cast<unsigned>(blocks)), dim3(32 * kJoinWarps), 0, stream, p)
            : launch_pdl(join_kernel<R, true>, by, dim3(32 * kJoinWarps), 0, stream, p);
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
  // Time is counted in 32 bits, by the most tiles that sequences can have: of a longer prefix than the table has room for there are none.
  const long long most = std::min<long long>(static_cast<long long>(a.max_prefix) + a.m, static_cast<long long>(a.max_blocks) * a.block_size);
  if (((most + BK - 1) / BK + kBegin) * a.B * a.Hkv > INT32_MAX) return TS_ERR_UNSUPPORTED;
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
  p.scale_log2 = 0.25f * a.scale * kLog2e;
  const float q_end = kMostQ / a.scale;  // (an infinity for the least scales)
  std::memcpy(&p.q_end, &q_end, sizeof p.q_end);
  CUtensorMap mk, mv;
  if (!encode_map(&mk, a.k_cache, a.num_blocks, a.Hkv, a.block_size) || !encode_map(&mv, a.v_cache, a.num_blocks, a.Hkv, a.block_size))
    return TS_ERR_CUDA;
  switch (pl.R) {
    case 16: return launch<16, 1>(p, mk, mv, stream);  // (up to 32 rows a thread has one key)
    case 32: return launch<32, 1>(p, mk, mv, stream);
    default:
      return a.scale_block >= 16  ? launch<128, 16>(p, mk, mv, stream)
             : a.scale_block >= 4 ? launch<128, 4>(p, mk, mv, stream)
                                  : launch<128, 1>(p, mk, mv, stream);
  }
}

}  // namespace ts
