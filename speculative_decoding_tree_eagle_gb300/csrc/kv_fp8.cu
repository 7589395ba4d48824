// The paged cache in 8 bits: ts_kv_write_fp8, ts_kv_read_fp8, ts_kv_commit_fp8.
//
// Definition (fp8_cache.cuh has the format).  A write of rows into positions start .. end - 1 quantises every block of
// sb positions that gets a new row, for each KV head, K and V apart, over its kept rows (below start; code * old scale)
// and its new ones:
//   2^e = the smallest power of two in [2^-40, 2^40] with max |value| <= 448 * 2^e,   code = e4m3(value * 2^-e)
// so a block's scale depends on the rows it holds alone: rejected rows that had raised it are forgotten by the next
// write.  Rows behind the last new one keep their bytes and lose their meaning.
//
// What bounds them: a prompt's write reads 2 or 4 bytes and writes one per element, a read the other way round: HBM.
// The writes of single tokens and trees, and the commit, are latency: table entry -> rows -> maximum -> codes.
//
// Measured on the device (GB300, replayed from a graph, 8 heads of 128): a prompt of 4 x 32768 bf16 rows 123 us (93% of the
// copy rate), of 2 x 32768 fp32 rows 102 (95%), 60-node trees of 16 sequences 4.0,
// one token of each of 64 sequences in 64-token blocks 4.8 (it reads its block's kept rows); a read of 2 x 8192 rows into bf16 18
// (82%), of 16 x 64 into fp32 5.1; a commit of at most 7 rows of 16 sequences 6.0, of 16 rows of 64 sequences in 64-token blocks 10.8.
// Head dims that are not a power of two go element by element: the same prompt with d = 96 747 us, with d = 192 1197 (11% and 14% of the
// copy rate).
#include <algorithm>
#include <type_traits>

#include "fp8_cache.cuh"
#include "internal.h"

namespace ts {
namespace {

// Threads of a CTA whose items have W warps each, and CTAs per SM that its registers are to leave room for.  More CTAs of fewer
// threads keep more reads in flight while others wait for their maximum: a prompt of 4 x 32768 bf16 rows took 144 us with 256
// threads and what registers the compiler liked (75), 140 with 128, 127 with eight such CTAs (64 registers), 130 with seven or nine
// (and 122 with multiplications in place of the item's five divisions).
__host__ __device__ constexpr int write_threads(int W) { return W > 4 ? 32 * W : 128; }
template <typename T>
__host__ __device__ constexpr int write_ctas(int W) { return (sizeof(T) == 2 ? 1024 : 640) / write_threads(W); }
constexpr int kAnyThreads = 256;
constexpr int kChunk = 8;     // elements that a thread loads at once (16 bytes of bf16, 8 codes)
constexpr int kHeld = 8;      // chunks that a thread holds between the maximum and the codes

// x / d for 0 <= x < 2^31 as a multiplication (Granlund and Montgomery, "Division by invariant integers using multiplication",
// 1994): with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1 the quotient is (x m / 2^32 + x) / 2^s.  (Six divisions a
// thread took a third of a read's instructions, five a warp more than the rest of a write with four tokens to a scale.)
struct Divide {
  uint32_t m, s, d;
  Divide() = default;
  explicit Divide(int by) : d(static_cast<uint32_t>(by)) {
    s = 0;
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ int quotient(int x) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(x), m) + static_cast<uint32_t>(x)) >> s);
  }
};

struct Side {                 // K or V
  const void* src;            // [B, n, Hkv, d], element strides below
  long long sb_, sn, sh;
  uint8_t* cache;
  float* scale;
};
struct WriteParams {
  Side side[2];
  const int32_t* table;
  const int32_t* start_len;
  const int32_t* length;
  int32_t* status;
  int B, n, Hkv, d, bs, sb, nsb, max_blocks, num_blocks, blocks;  // blocks: that n rows can touch
  Divide by_head, by_page, by_block;
};

// One (K or V, sequence, block, head) of a write.
struct Item {
  bool live;
  int first, rows_kept, rows_end;  // block's first position; rows [0, kept) are kept, [kept, end) new
  const char* src;                 // the block's first row (it may lie before the tensor where that row is kept)
  uint8_t* codes;
  float* scale;
};

// Block i, head h of sequence b.
template <typename T>
__device__ __forceinline__ Item item_of(const WriteParams& p, const Side& side, int b, int i, int h) {
  Item it;
  it.live = false;
  if (i >= p.blocks) return it;
  const int start = p.start_len[b], len = p.length != nullptr ? p.length[b] : p.n;
  const long long end = static_cast<long long>(start) + len;
  if (start < 0 || len < 0 || len > p.n || end > min(static_cast<long long>(p.max_blocks) * p.bs, static_cast<long long>(INT32_MAX))) {
    if (i == 0) report(p.status, TS_ERR_DEVICE_CHECK);
    return it;
  }
  const long long first_at = (static_cast<long long>(p.by_block.quotient(start)) + i) * p.sb;
  if (len == 0 || first_at >= end) return it;
  const int first = static_cast<int>(first_at), lp = p.by_page.quotient(first);
  const int page = p.table[static_cast<long long>(b) * p.max_blocks + lp];
  if (page < 0 || page >= p.num_blocks) {
    report(p.status, TS_ERR_DEVICE_CHECK);
    return it;
  }
  it.live = true;
  it.first = first;
  it.rows_kept = max(0, start - first);
  it.rows_end = static_cast<int>(min(static_cast<long long>(p.sb), end - first));
  const int row = first - lp * p.bs;
  const long long head = static_cast<long long>(page) * p.Hkv + h;
  it.codes = side.cache + (head * p.bs + row) * p.d;
  it.scale = side.scale + head * p.nsb + p.by_block.quotient(row);
  it.src = static_cast<const char*>(side.src) + (static_cast<long long>(b) * side.sb_ + static_cast<long long>(first - start) * side.sn +
                                                 static_cast<long long>(h) * side.sh) * static_cast<long long>(sizeof(T));
  return it;
}

template <typename T>
struct Held {};  // kChunk elements as they lie in memory
template <>
struct Held<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const void* p) { w = __ldg(static_cast<const uint4*>(p)); }
  __device__ void keep(uint2 c) { w.x = c.x, w.y = c.y; }
  __device__ uint2 kept() const { return make_uint2(w.x, w.y); }
  __device__ float largest() const {  // (max passes over a NaN)
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);
  }
  __device__ void values(float (&v)[8]) const {
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
  }
};
template <>
struct Held<float> {
  float4 a, b;
  __device__ void keep(uint2 c) { a.x = __uint_as_float(c.x), a.y = __uint_as_float(c.y); }
  __device__ uint2 kept() const { return make_uint2(__float_as_uint(a.x), __float_as_uint(a.y)); }
  __device__ float largest() const {
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                 fmaxf(fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))), 0.f));
  }
  __device__ void load(const void* p) {
    a = __ldg(static_cast<const float4*>(p));
    b = __ldg(static_cast<const float4*>(p) + 1);
  }
  __device__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

__device__ __forceinline__ void decode8(uint2 c, float (&v)[8]) {
  const float2 a = decode_e4m3x2(c.x), b = decode_e4m3x2(c.x >> 16), e = decode_e4m3x2(c.y), f = decode_e4m3x2(c.y >> 16);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = e.x, v[5] = e.y, v[6] = f.x, v[7] = f.y;
}
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float by) {
  uint2 c;
  c.x = encode_e4m3x2(v[0] * by, v[1] * by) | (encode_e4m3x2(v[2] * by, v[3] * by) << 16);
  c.y = encode_e4m3x2(v[4] * by, v[5] * by) | (encode_e4m3x2(v[6] * by, v[7] * by) << 16);
  return c;
}
__device__ __forceinline__ float largest_code(uint2 c) {  // (NaN passed over)
  float v[8], m = 0.f;
  decode8(c, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  return m;
}

// W warps per item, kChunk elements a load (d, strides and addresses are multiples of it).  The W * 32 threads cover whole rows (d / kChunk
// divides their number), so a thread stays in its columns and no load costs a division.  Where the block fits in kHeld chunks per
// thread the rows stay in registers between the maximum and the codes, otherwise they are read twice.
template <typename T, int W, bool HOLD>
__global__ void __launch_bounds__(write_threads(W), write_ctas<T>(W)) write_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kItems = write_threads(W) / (32 * W);  // of a CTA
  __shared__ float s_max[kItems * W];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / W, part = (warp % W) * 32 + lane;  // item of this CTA, thread of the item
  const Side& side = p.side[blockIdx.z];
  const int x = blockIdx.x * kItems + sub, block = p.by_head.quotient(x);
  const Item it = item_of<T>(p, side, blockIdx.y, block, x - block * p.Hkv);
  if (W == 1 && !it.live) return;
  const int per_row = p.d / kChunk, step = 32 * W / per_row, r0 = part / per_row, col = (part - r0 * per_row) * kChunk;
  const int kept = it.live ? it.rows_kept : 0, end = it.live ? it.rows_end : 0;
  const float old = kept > 0 ? scale_in_range(*it.scale) : 1.f;
  const char* src = it.src + (static_cast<long long>(r0) * side.sn + col) * static_cast<long long>(sizeof(T));
  const long long src_step = static_cast<long long>(step) * side.sn * static_cast<long long>(sizeof(T));
  uint8_t* codes = it.codes + r0 * p.d + col;
  const int codes_step = step * p.d;
  float amax = 0.f, v[8];
  Held<T> held[HOLD ? kHeld : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int r = r0 + u * step;
      if (r >= kept && r < end) held[u].load(src + u * src_step);
      else if (r < end) held[u].keep(*reinterpret_cast<const uint2*>(codes + u * codes_step));
    }
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int r = r0 + u * step;
      if (r >= kept && r < end) amax = fmaxf(amax, held[u].largest());
      else if (r < end) amax = fmaxf(amax, largest_code(held[u].kept()) * old);
    }
  } else {
    for (int r = r0; r < end; r += step) {
      if (r >= kept) {
        held[0].load(src + (r - r0) / step * src_step);
        amax = fmaxf(amax, held[0].largest());
      } else {
        amax = fmaxf(amax, largest_code(*reinterpret_cast<const uint2*>(codes + (r - r0) / step * codes_step)) * old);
      }
    }
  }
  // (magnitudes order as their bits do)
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if constexpr (W > 1) {
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) amax = fmaxf(amax, s_max[sub * W + w]);
    if (!it.live) return;
  }
  const int e = scale_exponent(amax);
  const float inv = pow2(-e);
  const float again = old * inv;  // from kept codes to codes
  if constexpr (HOLD) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int r = r0 + u * step;
      if (r >= end || (r < kept && again == 1.f)) continue;
      if (r < kept) decode8(held[u].kept(), v);
      else held[u].values(v);
      *reinterpret_cast<uint2*>(codes + u * codes_step) = encode8(v, r < kept ? again : inv);
    }
  } else {
    for (int r = r0; r < end; r += step) {
      if (r < kept && again == 1.f) continue;
      uint2* to = reinterpret_cast<uint2*>(codes + (r - r0) / step * codes_step);
      if (r < kept) {
        decode8(*to, v);
      } else {
        held[0].load(src + (r - r0) / step * src_step);
        held[0].values(v);
      }
      *to = encode8(v, r < kept ? again : inv);
    }
  }
  if (part == 0) *it.scale = pow2(e);
}

__device__ __forceinline__ float element(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float element(const float* p) { return *p; }

// Blocks smaller than what a warp holds (kHeld chunks per thread: `run` rows): a warp takes a run of positions with all their blocks, so
// its loads are as many as for larger blocks.  Thread and rows as in write_kernel; a block is either some of a thread's chunks and all
// threads, or one chunk of some neighbouring threads.  (A warp per block: 4 x 32768 bf16 rows with four tokens
// to a scale 276 us, 164 by runs; 2 x 32768 with a scale for each 497 and 101.  Seven CTAs to an SM, 72 registers: with eight it spills,
// 185 us.)
template <typename T>
__global__ void __launch_bounds__(write_threads(1), sizeof(T) == 2 ? 7 : 4) write_runs_kernel(const __grid_constant__ WriteParams p) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const Side& side = p.side[blockIdx.z];
  const int x = blockIdx.x * (write_threads(1) / 32) + warp, i = p.by_head.quotient(x), h = x - i * p.Hkv;
  const int per_row = p.d / kChunk, step = 32 / per_row, run = kHeld * step, r0 = lane / per_row, col = (lane - r0 * per_row) * kChunk;
  if (i >= p.blocks) return;
  const int start = p.start_len[b], len = p.length != nullptr ? p.length[b] : p.n;
  const long long end = static_cast<long long>(start) + len;
  if (start < 0 || len < 0 || len > p.n || end > min(static_cast<long long>(p.max_blocks) * p.bs, static_cast<long long>(INT32_MAX))) {
    if (i == 0) report(p.status, TS_ERR_DEVICE_CHECK);
    return;
  }
  const long long first_at = (static_cast<long long>(start / run) + i) * run;
  if (len == 0 || first_at >= end) return;
  const int first = static_cast<int>(first_at), lp = p.by_page.quotient(first);
  const int page = p.table[static_cast<long long>(b) * p.max_blocks + lp];
  if (page < 0 || page >= p.num_blocks) {
    report(p.status, TS_ERR_DEVICE_CHECK);
    return;
  }
  // rows [low, kept) are kept ones of the block that `start` lies in, [kept, top) are new
  const int low = max(0, p.by_block.quotient(start) * p.sb - first), kept = max(0, start - first);
  const int top = static_cast<int>(min(static_cast<long long>(run), end - first));
  const int at = first - lp * p.bs;
  const long long head = static_cast<long long>(page) * p.Hkv + h;
  uint8_t* codes = side.cache + (head * p.bs + at + r0) * p.d + col;
  float* scale = side.scale + head * p.nsb + p.by_block.quotient(at);
  const char* src = static_cast<const char*>(side.src) +
                    (static_cast<long long>(b) * side.sb_ + static_cast<long long>(first - start + r0) * side.sn +
                     static_cast<long long>(h) * side.sh + col) * static_cast<long long>(sizeof(T));
  const long long src_step = static_cast<long long>(step) * side.sn * static_cast<long long>(sizeof(T));
  const int codes_step = step * p.d;
  const float old = kept > low ? scale_in_range(scale[p.by_block.quotient(low)]) : 1.f;
  Held<T> held[kHeld];
  float m[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int r = r0 + u * step;
    if (r >= kept && r < top) held[u].load(src + u * src_step);
    else if (r >= low && r < top) held[u].keep(*reinterpret_cast<const uint2*>(codes + u * codes_step));
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int r = r0 + u * step;
    m[u] = r >= kept && r < top ? held[u].largest() : r >= low && r < top ? largest_code(held[u].kept()) * old : 0.f;
  }
  // the largest of each block: among a thread's chunks, then among threads (magnitudes order as their bits do)
#pragma unroll
  for (int o = 1; o < kHeld; o <<= 1) {
    if (o * step < p.sb) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if ((u & o) == 0) m[u] = m[u + o] = fmaxf(m[u], m[u + o]);
    }
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    if (p.sb >= step) {
      m[u] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m[u])));
    } else {
      for (int o = per_row * p.sb / 2; o > 0; o >>= 1) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
    }
  }
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int r = r0 + u * step;
    if (r < low || r >= top) continue;
    const int e = scale_exponent(m[u]);
    const float inv = pow2(-e), again = old * inv;  // from kept codes to codes
    if (r >= kept || again != 1.f) {
      float v[8];
      if (r < kept) decode8(held[u].kept(), v);
      else held[u].values(v);
      *reinterpret_cast<uint2*>(codes + u * codes_step) = encode8(v, r < kept ? again : inv);
    }
    if (col == 0 && (r & (p.sb - 1)) == 0) scale[p.by_block.quotient(r)] = pow2(e);
  }
}

// Any head dim, strides and alignment: a CTA per item, element by element, the rows read twice.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) write_any_kernel(const __grid_constant__ WriteParams p) {
  __shared__ float s_max[kAnyThreads / 32];
  pdl_wait();
  const Side& side = p.side[blockIdx.z];
  const int block = blockIdx.x / p.Hkv;
  const Item it = item_of<T>(p, side, blockIdx.y, block, blockIdx.x - block * p.Hkv);
  if (!it.live) return;
  const int total = it.rows_end * p.d;
  const float old = it.rows_kept > 0 ? scale_in_range(*it.scale) : 1.f;
  const T* src = reinterpret_cast<const T*>(it.src);
  auto value = [&](int x, bool& kept) {
    const int r = x / p.d;
    kept = r < it.rows_kept;
    return kept ? decode_e4m3(it.codes[x]) : element(src + static_cast<long long>(r) * side.sn + (x - r * p.d));
  };
  float amax = 0.f;
  bool kept;
  for (int x = threadIdx.x; x < total; x += kAnyThreads) {
    const float v = fabsf(value(x, kept));
    amax = fmaxf(amax, kept ? v * old : v);
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAnyThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  const int e = scale_exponent(amax);
  const float inv = pow2(-e);
  for (int x = threadIdx.x; x < total; x += kAnyThreads) {
    const float v = value(x, kept);
    it.codes[x] = static_cast<uint8_t>(encode_e4m3x2(kept ? v * (old * inv) : v * inv, 0.f) & 0xFFu);
  }
  if (threadIdx.x == 0) *it.scale = pow2(e);
}

// ---------------------------------------------------------------------------------------------- read
constexpr int kReadThreads = 256;

struct ReadParams {
  const uint8_t* cache[2];
  const float* scale[2];
  void* out[2];
  const int32_t* table;
  const int32_t* prefix_len;
  const int32_t* start_len;
  int32_t* status;
  int B, n, Hkv, d, bs, sb, max_blocks, num_blocks;
  Divide by_heads, by_row, by_page, by_block;  // chunks of a token, of a head's row; tokens of a page, of a scale
};

// Whether sequence b can be read; its positions start .. end - 1 exist.
__device__ __forceinline__ bool read_range(const ReadParams& p, int b, int& start, int& rows) {
  start = p.start_len != nullptr ? p.start_len[b] : 0;
  const int L = p.prefix_len[b];
  rows = 0;
  if (start < 0 || L < 0 || static_cast<long long>(L) > static_cast<long long>(p.max_blocks) * p.bs) return false;
  rows = max(0, min(p.n, L - start));
  return true;
}

// A thread per N codes of a row: N values of type T out (N = 16: one 16-byte load; N = 1: any head dim and alignment), kAtOnce rows
// apart in flight, as each is three dependent loads (table, codes and scale).
constexpr int kAtOnce = 2;
template <typename T, int N>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_wait();
  const int b = blockIdx.y, kv = blockIdx.z;
  int start, rows;
  if (!read_range(p, b, start, rows) && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, TS_ERR_DEVICE_CHECK);
  const int per = p.d / N, heads = p.Hkv * per, nsb = p.bs / p.sb;
  const int total = p.n * heads, step = gridDim.x * kReadThreads;  // (checked on the host to stay below 2^31 with all steps)
  T* out = static_cast<T*>(p.out[kv]) + static_cast<long long>(b) * total * N;
  const int32_t* table = p.table + static_cast<long long>(b) * p.max_blocks;
  for (int x0 = blockIdx.x * kReadThreads + threadIdx.x; x0 < total; x0 += kAtOnce * step) {
    uint4 w[kAtOnce];
    float s[kAtOnce];
    int page[kAtOnce], pos[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int x = x0 + u * step, t = p.by_heads.quotient(x);
      pos[u] = start + t;
      page[u] = x < total && t < rows ? table[p.by_page.quotient(pos[u])] : -1;
      if (x < total && t < rows && (page[u] < 0 || page[u] >= p.num_blocks)) {
        report(p.status, TS_ERR_DEVICE_CHECK);
        page[u] = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      w[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.f;
      if (page[u] >= 0) {
        const int rest = x0 + u * step - (pos[u] - start) * heads, h = p.by_row.quotient(rest), c = rest - h * per;
        const int row = pos[u] - p.by_page.quotient(pos[u]) * p.bs;
        const long long head = static_cast<long long>(page[u]) * p.Hkv + h;
        const uint8_t* from = p.cache[kv] + (head * p.bs + row) * p.d + c * N;
        s[u] = p.scale[kv][head * nsb + p.by_block.quotient(row)];
        if constexpr (N == 16) w[u] = *reinterpret_cast<const uint4*>(from);
        else w[u].x = *from;
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int x = x0 + u * step;
      if (x >= total) break;
      const float f = scale_in_range(s[u]);  // (codes of 0 where there is nothing to read)
      if constexpr (N == 1) {
        const float v = decode_e4m3(w[u].x) * f;
        if constexpr (sizeof(T) == 2) out[x] = __float2bfloat16_rn(v);
        else out[x] = v;
      } else {
        const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = decode_e4m3x2(in[j]), hi = decode_e4m3x2(in[j] >> 16);
          v[4 * j] = lo.x * f, v[4 * j + 1] = lo.y * f, v[4 * j + 2] = hi.x * f, v[4 * j + 3] = hi.y * f;
        }
        if constexpr (sizeof(T) == 2) {
          uint4* to = reinterpret_cast<uint4*>(out + static_cast<long long>(x) * 16);
          to[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          to[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                             pack_bf16x2(v[14], v[15]));
        } else {
          float4* to = reinterpret_cast<float4*>(out + static_cast<long long>(x) * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------- commit
constexpr int kCommitThreads = 256;
constexpr int kMaxPages = TS_MAX_NODES + 2;  // pages a tree of <= 256 nodes can touch (any page size)

struct CommitParams {
  uint8_t* cache[2];
  float* scale[2];
  const int32_t* table;
  const int32_t* prefix_len;
  const int32_t* accept_path;
  const int32_t* accept_len;
  int32_t* table_out;
  int32_t* prefix_out;
  int32_t* freed;
  int32_t* freed_count;
  int32_t* status;
  int B, m, Hkv, d, bs, sb, max_blocks, num_blocks;
  bool in_place;  // a table or length is written over its input: in a launch of its own, after the rows have read it
};

// The contract of ts_kv_commit, checked by the whole CTA for sequence b; the path and the ids of the pages that tree
// positions touch go to shared memory.
struct Commit {
  bool ok;
  int L, a, p0, n_keep, n_used;
};
__device__ __forceinline__ Commit commit_of(const CommitParams& p, int b, int* s_path, int* s_page) {
  Commit c;
  c.L = p.prefix_len[b];
  c.a = p.accept_len[b];
  const long long used = c.L >= 0 ? (static_cast<long long>(c.L) + p.m + p.bs - 1) / p.bs : 0;
  bool bad = c.L < 0 || c.L > INT32_MAX - TS_MAX_NODES || c.a < 1 || c.a > p.m || used > p.max_blocks;
  c.n_used = bad ? 0 : static_cast<int>(used);
  c.n_keep = bad ? 0 : static_cast<int>((static_cast<long long>(c.L) + c.a + p.bs - 1) / p.bs);
  c.p0 = bad ? 0 : c.L / p.bs;
  bad = bad || c.n_used - c.p0 > kMaxPages;
  if (!bad) {
    for (int j = threadIdx.x; j < c.a; j += blockDim.x) {
      const int32_t* path = p.accept_path + static_cast<long long>(b) * p.m;
      const int pj = path[j];
      s_path[j] = pj;
      if (j == 0 ? pj != 0 : (pj >= p.m || pj <= path[j - 1])) bad = true;
    }
    // (by distances from p0: positions and cells may lie just below 2^31)
    for (int i = threadIdx.x; i < c.n_used - c.p0; i += blockDim.x) {
      const int pg = p.table[static_cast<long long>(b) * p.max_blocks + c.p0 + i];
      s_page[i] = pg;
      if (pg < 0 || pg >= p.num_blocks) bad = true;
    }
  }
  c.ok = !__syncthreads_or(bad);
  return c;
}

// Tables, lengths and the released pages of sequence b, by the whole CTA.
__device__ void commit_tables(const CommitParams& p, int b, const Commit& c, const int* s_page) {
  const long long o = static_cast<long long>(b) * p.max_blocks;
  // (unsigned: a step behind the last cell does not wrap, nor does a cell and a page's number)
  const uint32_t cells = p.max_blocks, keep = c.n_keep, used = c.n_used;
  for (uint32_t i = threadIdx.x; i < cells; i += kCommitThreads) {
    const uint32_t k = i + keep;
    p.freed[o + i] = c.ok && k < used ? s_page[k - c.p0] : -1;
    const bool gone = c.ok && i >= keep && i < used;
    if (gone) p.table_out[o + i] = -1;
    else if (p.table_out != p.table) p.table_out[o + i] = p.table[o + i];
  }
  if (threadIdx.x == 0) {
    p.freed_count[b] = c.ok ? c.n_used - c.n_keep : 0;
    p.prefix_out[b] = c.ok ? c.L + c.a : c.L;
    if (!c.ok) report(p.status, TS_ERR_DEVICE_CHECK);
  }
}

// N codes as they are loaded, and what is done to them.
template <int N>
struct Codes;
template <>
struct Codes<16> {
  uint4 w;
  __device__ float largest() const {
    return fmaxf(largest_code(make_uint2(w.x, w.y)), largest_code(make_uint2(w.z, w.w)));
  }
  __device__ void times(float f) {
    float v[8];
    decode8(make_uint2(w.x, w.y), v);
    const uint2 a = encode8(v, f);
    decode8(make_uint2(w.z, w.w), v);
    const uint2 b = encode8(v, f);
    w = make_uint4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Codes<4> {
  uint32_t w;
  __device__ float largest() const {
    const float2 a = decode_e4m3x2(w), b = decode_e4m3x2(w >> 16);
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))), 0.f);
  }
  __device__ void times(float f) {
    const float2 a = decode_e4m3x2(w), b = decode_e4m3x2(w >> 16);
    w = encode_e4m3x2(a.x * f, a.y * f) | (encode_e4m3x2(b.x * f, b.y * f) << 16);
  }
};
template <>
struct Codes<1> {
  uint8_t w;
  __device__ float largest() const { return fmaxf(fabsf(decode_e4m3(w)), 0.f); }
  __device__ void times(float f) { w = static_cast<uint8_t>(encode_e4m3x2(decode_e4m3(w) * f, 0.f)); }
};

// A CTA per (sequence, KV head, K or V).  The accepted rows' codes and scales are staged in shared memory, so every row is
// read before any is written; then a team of threads per block quantises its kept and its new rows: a warp, or the whole CTA (WHOLE) for
// blocks of more than 2048 codes, of which a path touches one or two (64 x 128 codes by a warp: 11 of 19 us).
template <int N, bool WHOLE>  // N codes a load: 16, 4 or 1
__global__ void __launch_bounds__(kCommitThreads) commit_rows_kernel(const __grid_constant__ CommitParams p) {
  extern __shared__ __align__(16) unsigned char s_rows[];
  __shared__ int s_path[TS_MAX_NODES];
  __shared__ int s_page[kMaxPages];
  __shared__ float s_scale[TS_MAX_NODES];
  __shared__ float s_max[kCommitThreads / 32];
  using Word = Codes<N>;
  pdl_wait();
  const int b = blockIdx.y, h = blockIdx.x >> 1, kv = blockIdx.x & 1;
  const Commit c = commit_of(p, b, s_path, s_page);
  if (!p.in_place && blockIdx.x == 0) commit_tables(p, b, c, s_page);
  if (!c.ok) return;
  uint8_t* cache = p.cache[kv];
  float* scale = p.scale[kv];
  const int nsb = p.bs / p.sb, per = p.d / N;
  auto head_of = [&](int pos) { return static_cast<long long>(s_page[pos / p.bs - c.p0]) * p.Hkv + h; };
  for (int x = threadIdx.x; x < c.a * per; x += kCommitThreads) {
    const int j = x / per, q = x - j * per, pos = c.L + s_path[j];
    reinterpret_cast<Word*>(s_rows)[x] =
        *reinterpret_cast<const Word*>(cache + (head_of(pos) * p.bs + pos % p.bs) * p.d + q * N);
    if (q == 0) s_scale[j] = scale_in_range(scale[head_of(pos) * nsb + pos % p.bs / p.sb]);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = WHOLE ? 0 : warp, teams = WHOLE ? 1 : kCommitThreads / 32;
  const int me = WHOLE ? threadIdx.x : lane, size = WHOLE ? kCommitThreads : 32;
  const int blk0 = c.L / p.sb, blocks = (c.L + c.a - 1) / p.sb - blk0 + 1;
  for (int i = team; i < blocks; i += teams) {
    const int first = (blk0 + i) * p.sb, kept = max(0, c.L - first), end = min(p.sb, c.L + c.a - first);
    const long long head = head_of(max(first, c.L));
    Word* codes = reinterpret_cast<Word*>(cache + (head * p.bs + first % p.bs) * p.d);
    float* sc = scale + head * nsb + first % p.bs / p.sb;
    const float old = kept > 0 ? scale_in_range(*sc) : 1.f;
    const Word* rows = reinterpret_cast<const Word*>(s_rows) + (first - c.L) * per;
    float amax = 0.f;
    for (int x = me; x < end * per; x += size) {
      const int r = x / per;
      amax = fmaxf(amax, r < kept ? codes[x].largest() * old : rows[x].largest() * s_scale[first + r - c.L]);
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if constexpr (WHOLE) {
      __syncthreads();  // (the last block's maxima have been read; everyone has the old scale)
      if (lane == 0) s_max[warp] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kCommitThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
    }
    const int e = scale_exponent(amax);
    const float inv = pow2(-e);
    for (int x = me; x < end * per; x += size) {
      const int r = x / per;
      if (r < kept && old * inv == 1.f) continue;
      Word w = r < kept ? codes[x] : rows[x];
      w.times((r < kept ? old : s_scale[first + r - c.L]) * inv);
      codes[x] = w;
    }
    __syncwarp();
    if (me == 0) *sc = pow2(e);
  }
}

// The tables of an update in place, after the rows have moved: a CTA per sequence.
__global__ void __launch_bounds__(kCommitThreads) commit_table_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int s_path[TS_MAX_NODES];
  __shared__ int s_page[kMaxPages];
  pdl_wait();
  const Commit c = commit_of(p, blockIdx.x, s_path, s_page);
  commit_tables(p, blockIdx.x, c, s_page);
}

// Blocks (of K and V) from which a warp takes a run of them: below, a call is latency, which a warp per block spreads (with four
// tokens to a scale one token of 64 sequences 3.6 us for 4.4, trees of 60 nodes of 16 4.6 for 5.5).  Half a run to a block is
// faster by blocks too (165 for 185 us).
constexpr long long kManyBlocks = 32768;

template <typename T>
cudaError_t launch_write(const WriteParams& p, bool wide, cudaStream_t stream) {
  const int chunks = (p.sb * p.d + kChunk - 1) / kChunk, held = 32 * kHeld, items = p.blocks * p.Hkv;
  if (!wide) return launch_pdl(write_any_kernel<T>, dim3(items, p.B, 2), dim3(kAnyThreads), 0, stream, p);
  auto launch = [&](auto kernel, int w) {
    const int each = write_threads(w) / (32 * w);
    return launch_pdl(kernel, dim3((items + each - 1) / each, p.B, 2), dim3(write_threads(w)), 0, stream, p);
  };
  // (d is a power of two here, a run one too, and what divides it)
  const int run = held * kChunk / p.d;
  if (2 * p.sb < run && run % p.sb == 0 && p.bs % run == 0 && 2LL * items * p.B >= kManyBlocks) {
    WriteParams q = p;
    q.blocks = static_cast<int>((static_cast<long long>(p.n) + 2LL * run - 2) / run);  // (runs, here)
    const int each = write_threads(1) / 32;
    return launch_pdl(write_runs_kernel<T>, dim3((q.blocks * q.Hkv + each - 1) / each, q.B, 2), dim3(write_threads(1)), 0, stream, q);
  }
  if (chunks <= held) return launch(write_kernel<T, 1, true>, 1);
  if (chunks <= 2 * held) return launch(write_kernel<T, 2, true>, 2);
  if (chunks <= 4 * held) return launch(write_kernel<T, 4, true>, 4);
  if (chunks <= 8 * held) return launch(write_kernel<T, 8, true>, 8);
  return launch(write_kernel<T, 8, false>, 8);
}

}  // namespace

int kv_write_fp8_launch(const Fp8WriteCall& c, cudaStream_t stream) {
  WriteParams p;
  p.side[0] = Side{c.k, c.k_stride[0], c.k_stride[1], c.k_stride[2], static_cast<uint8_t*>(c.k_cache), c.k_scale};
  p.side[1] = Side{c.v, c.v_stride[0], c.v_stride[1], c.v_stride[2], static_cast<uint8_t*>(c.v_cache), c.v_scale};
  p.table = c.block_table;
  p.start_len = c.start_len;
  p.length = c.length;
  p.status = c.dev_status;
  p.B = c.B, p.n = c.n, p.Hkv = c.Hkv, p.d = c.d, p.bs = c.block_size, p.sb = c.scale_block;
  p.nsb = c.block_size / c.scale_block, p.max_blocks = c.max_blocks, p.num_blocks = c.num_blocks;
  p.by_head = Divide(c.Hkv), p.by_page = Divide(c.block_size), p.by_block = Divide(c.scale_block);
  p.blocks = static_cast<int>((static_cast<long long>(c.n) + 2LL * c.scale_block - 2) / c.scale_block);
  if (static_cast<long long>(p.blocks) * c.Hkv > INT32_MAX - 8) return TS_ERR_UNSUPPORTED;
  const size_t size = c.dt == TS_BF16 ? 2 : 4;
  bool wide = c.d % kChunk == 0 && 32 % (c.d / kChunk) == 0;  // (a head dim of 8, 16, 32, 64, 128 or 256)
  for (const Side& s : p.side) {
    wide = wide && reinterpret_cast<uintptr_t>(s.src) % 16 == 0 && reinterpret_cast<uintptr_t>(s.cache) % 8 == 0;
    for (long long st : {s.sb_, s.sn, s.sh}) wide = wide && st * static_cast<long long>(size) % 16 == 0;
  }
  const cudaError_t e = c.dt == TS_BF16 ? launch_write<__nv_bfloat16>(p, wide, stream) : launch_write<float>(p, wide, stream);
  count_launches(1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

int kv_read_fp8_launch(const Fp8ReadCall& c, cudaStream_t stream, int num_sms) {
  ReadParams p;
  p.cache[0] = static_cast<const uint8_t*>(c.k_cache), p.cache[1] = static_cast<const uint8_t*>(c.v_cache);
  p.scale[0] = c.k_scale, p.scale[1] = c.v_scale;
  p.out[0] = c.k, p.out[1] = c.v;
  p.table = c.block_table, p.prefix_len = c.prefix_len, p.start_len = c.start_len, p.status = c.dev_status;
  p.B = c.B, p.n = c.n, p.Hkv = c.Hkv, p.d = c.d, p.bs = c.block_size, p.sb = c.scale_block;
  p.max_blocks = c.max_blocks, p.num_blocks = c.num_blocks;
  bool wide = c.d % 16 == 0;
  for (const void* x : {c.k_cache, c.v_cache, static_cast<const void*>(c.k), static_cast<const void*>(c.v)})
    wide = wide && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  const long long total = static_cast<long long>(c.n) * c.Hkv * (c.d / (wide ? 16 : 1));
  p.by_heads = Divide(c.Hkv * (c.d / (wide ? 16 : 1))), p.by_row = Divide(c.d / (wide ? 16 : 1));
  p.by_page = Divide(c.block_size), p.by_block = Divide(c.scale_block);
  // sixteen CTAs per SM at most, each thread with kAtOnce chunks where there are as many
  const long long most = std::max(1LL, (16LL * num_sms + 2LL * c.B - 1) / (2LL * c.B));
  const long long want = (total + kReadThreads * kAtOnce - 1) / (kReadThreads * kAtOnce);
  const unsigned gx = static_cast<unsigned>(std::max(1LL, std::min(want, most)));
  if (total + 2LL * kAtOnce * gx * kReadThreads > INT32_MAX) return TS_ERR_UNSUPPORTED;
  const dim3 grid(gx, c.B, 2), block(kReadThreads);
  cudaError_t e;
  if (c.dt == TS_BF16)
    e = wide ? launch_pdl(read_kernel<__nv_bfloat16, 16>, grid, block, 0, stream, p)
             : launch_pdl(read_kernel<__nv_bfloat16, 1>, grid, block, 0, stream, p);
  else
    e = wide ? launch_pdl(read_kernel<float, 16>, grid, block, 0, stream, p)
             : launch_pdl(read_kernel<float, 1>, grid, block, 0, stream, p);
  count_launches(1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

int kv_commit_fp8_launch(const Fp8CommitCall& c, cudaStream_t stream) {
  CommitParams p;
  p.cache[0] = static_cast<uint8_t*>(c.k_cache), p.cache[1] = static_cast<uint8_t*>(c.v_cache);
  p.scale[0] = c.k_scale, p.scale[1] = c.v_scale;
  p.table = c.block_table, p.prefix_len = c.prefix_len, p.accept_path = c.accept_path, p.accept_len = c.accept_len;
  p.table_out = c.block_table_out, p.prefix_out = c.prefix_len_out, p.freed = c.freed_blocks, p.freed_count = c.freed_count;
  p.status = c.dev_status;
  p.B = c.B, p.m = c.m, p.Hkv = c.Hkv, p.d = c.d, p.bs = c.block_size, p.sb = c.scale_block;
  p.max_blocks = c.max_blocks, p.num_blocks = c.num_blocks;
  p.in_place = c.block_table_out == c.block_table || c.prefix_len_out == c.prefix_len;
  const uintptr_t at = reinterpret_cast<uintptr_t>(c.k_cache) | reinterpret_cast<uintptr_t>(c.v_cache) | static_cast<uintptr_t>(c.d);
  const size_t smem = static_cast<size_t>(c.m) * c.d;  // at most 64 KB
  auto run = [&](auto kernel, std::atomic<uint64_t>& done) {
    cudaError_t e = once_per_device(done, [&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TS_MAX_NODES * 256);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(2 * c.Hkv, c.B), dim3(kCommitThreads), smem, stream, p);
  };
  static std::atomic<uint64_t> done[6]{};
  const bool whole = c.scale_block * c.d > 2048;
  cudaError_t e;
  if (at % 16 == 0) e = whole ? run(commit_rows_kernel<16, true>, done[0]) : run(commit_rows_kernel<16, false>, done[1]);
  else if (at % 4 == 0) e = whole ? run(commit_rows_kernel<4, true>, done[2]) : run(commit_rows_kernel<4, false>, done[3]);
  else e = whole ? run(commit_rows_kernel<1, true>, done[4]) : run(commit_rows_kernel<1, false>, done[5]);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  if (p.in_place) e = launch_pdl(commit_table_kernel, dim3(c.B), dim3(kCommitThreads), 0, stream, p);
  count_launches(p.in_place ? 2 : 1);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
