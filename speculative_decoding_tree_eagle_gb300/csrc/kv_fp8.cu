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
#include <algorithm>
#include <type_traits>

#include "fp8_cache.cuh"
#include "internal.h"

namespace ts {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kChunk = 8;     // elements that a thread loads at once (16 bytes of bf16, 8 codes)
constexpr int kHeld = 8;      // chunks that a thread holds between the maximum and the codes

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
  int B, n, Hkv, d, bs, sb, max_blocks, num_blocks, blocks;  // blocks: that n rows can touch
  long long items;                                           // 2 * B * blocks * Hkv
};

// One (K or V, sequence, block, head) of a write.
struct Item {
  bool live;
  int first, rows_kept, rows_end;  // block's first position; rows [0, kept) are kept, [kept, end) new
  const Side* side;
  int b, h;
  uint8_t* codes;                  // the block's first row
  float* scale;
};

__device__ __forceinline__ Item item_of(const WriteParams& p, long long idx) {
  Item it;
  it.live = false;
  if (idx >= p.items) return it;
  const int h = static_cast<int>(idx % p.Hkv);
  idx /= p.Hkv;
  const int i = static_cast<int>(idx % p.blocks);
  idx /= p.blocks;
  const int b = static_cast<int>(idx % p.B);
  it.side = &p.side[idx / p.B];
  it.b = b;
  it.h = h;
  const int start = p.start_len[b], len = p.length != nullptr ? p.length[b] : p.n;
  const long long end = static_cast<long long>(start) + len;
  if (start < 0 || len < 0 || len > p.n || end > min(static_cast<long long>(p.max_blocks) * p.bs, static_cast<long long>(INT32_MAX))) {
    if (i == 0) report(p.status, TS_ERR_DEVICE_CHECK);
    return it;
  }
  const long long first = (static_cast<long long>(start / p.sb) + i) * p.sb;
  if (len == 0 || first >= end) return it;
  const int lp = static_cast<int>(first / p.bs);
  const int page = p.table[static_cast<long long>(b) * p.max_blocks + lp];
  if (page < 0 || page >= p.num_blocks) {
    report(p.status, TS_ERR_DEVICE_CHECK);
    return it;
  }
  it.live = true;
  it.first = static_cast<int>(first);
  it.rows_kept = max(0, start - it.first);
  it.rows_end = static_cast<int>(min(static_cast<long long>(p.sb), end - first));
  const int row = it.first - lp * p.bs;
  const long long head = static_cast<long long>(page) * p.Hkv + h;
  it.codes = it.side->cache + (head * p.bs + row) * p.d;
  it.scale = it.side->scale + head * (p.bs / p.sb) + row / p.sb;
  return it;
}

template <typename T>
struct Held {};  // kChunk elements as they lie in memory
template <>
struct Held<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const void* p) { w = __ldg(static_cast<const uint4*>(p)); }
  __device__ void values(float (&v)[8]) const {
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
  }
};
template <>
struct Held<float> {
  float4 a, b;
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
__device__ __forceinline__ float absmax8(const float (&v)[8]) {  // (NaN passed over)
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  return m;
}

// W warps per item, kChunk elements a load (d, strides and addresses are multiples of it).  Where the block fits in
// kHeld chunks per thread the rows stay in registers between the maximum and the codes, otherwise they are read twice.
template <typename T, int W, bool HOLD>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const __grid_constant__ WriteParams p) {
  __shared__ float s_max[kWriteThreads / 32];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / W, part = (warp % W) * 32 + lane;  // item of this CTA, thread of the item
  const Item it = item_of(p, static_cast<long long>(blockIdx.x) * (kWriteThreads / (32 * W)) + sub);
  if (W == 1 && !it.live) return;
  const int cpr = p.d / kChunk, chunks = it.live ? it.rows_end * cpr : 0;
  const float old = it.live && it.rows_kept > 0 ? scale_in_range(*it.scale) : 1.f;
  const char* src = nullptr;
  if (it.live)
    src = static_cast<const char*>(it.side->src) +
          (static_cast<long long>(it.b) * it.side->sb_ + static_cast<long long>(it.first - p.start_len[it.b]) * it.side->sn +
           static_cast<long long>(it.h) * it.side->sh) * static_cast<long long>(sizeof(T));
  auto row_of = [&](int c) { return c / cpr; };
  auto from = [&](int c, int r) {
    return src + (static_cast<long long>(r) * it.side->sn + static_cast<long long>(c - r * cpr) * kChunk) * static_cast<long long>(sizeof(T));
  };
  float amax = 0.f, v[8];
  Held<T> held[HOLD ? kHeld : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int c = part + u * 32 * W;
      if (c < chunks) {
        const int r = row_of(c);
        if (r >= it.rows_kept) {
          held[u].load(from(c, r));
        } else {
          const uint2 k = *reinterpret_cast<const uint2*>(it.codes + static_cast<long long>(c) * kChunk);
          *reinterpret_cast<uint2*>(&held[u]) = k;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int c = part + u * 32 * W;
      if (c < chunks) {
        if (row_of(c) >= it.rows_kept) {
          held[u].values(v);
          amax = fmaxf(amax, absmax8(v));
        } else {
          decode8(*reinterpret_cast<const uint2*>(&held[u]), v);
          amax = fmaxf(amax, absmax8(v) * old);
        }
      }
    }
  } else {
    for (int c = part; c < chunks; c += 32 * W) {
      const int r = row_of(c);
      if (r >= it.rows_kept) {
        held[0].load(from(c, r));
        held[0].values(v);
        amax = fmaxf(amax, absmax8(v));
      } else {
        decode8(*reinterpret_cast<const uint2*>(it.codes + static_cast<long long>(c) * kChunk), v);
        amax = fmaxf(amax, absmax8(v) * old);
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
      const int c = part + u * 32 * W;
      if (c < chunks) {
        const bool kept = row_of(c) < it.rows_kept;
        if (kept && again == 1.f) continue;
        if (kept) decode8(*reinterpret_cast<const uint2*>(&held[u]), v);
        else held[u].values(v);
        *reinterpret_cast<uint2*>(it.codes + static_cast<long long>(c) * kChunk) = encode8(v, kept ? again : inv);
      }
    }
  } else {
    for (int c = part; c < chunks; c += 32 * W) {
      const int r = row_of(c);
      const bool kept = r < it.rows_kept;
      if (kept && again == 1.f) continue;
      uint8_t* to = it.codes + static_cast<long long>(c) * kChunk;
      if (kept) {
        decode8(*reinterpret_cast<const uint2*>(to), v);
      } else {
        held[0].load(from(c, r));
        held[0].values(v);
      }
      *reinterpret_cast<uint2*>(to) = encode8(v, kept ? again : inv);
    }
  }
  if (part == 0) *it.scale = pow2(e);
}

__device__ __forceinline__ float element(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float element(const float* p) { return *p; }

// Any head dim, strides and alignment: a CTA per item, element by element, the rows read twice.
template <typename T>
__global__ void __launch_bounds__(kWriteThreads) write_any_kernel(const __grid_constant__ WriteParams p) {
  __shared__ float s_max[kWriteThreads / 32];
  pdl_wait();
  const Item it = item_of(p, blockIdx.x);
  if (!it.live) return;
  const int total = it.rows_end * p.d;
  const float old = it.rows_kept > 0 ? scale_in_range(*it.scale) : 1.f;
  const T* src = static_cast<const T*>(it.side->src) + static_cast<long long>(it.b) * it.side->sb_ +
                 static_cast<long long>(it.first - p.start_len[it.b]) * it.side->sn + static_cast<long long>(it.h) * it.side->sh;
  auto value = [&](int x, bool& kept) {
    const int r = x / p.d;
    kept = r < it.rows_kept;
    return kept ? decode_e4m3(it.codes[x]) : element(src + static_cast<long long>(r) * it.side->sn + (x - r * p.d));
  };
  float amax = 0.f;
  bool kept;
  for (int x = threadIdx.x; x < total; x += kWriteThreads) {
    const float v = fabsf(value(x, kept));
    amax = fmaxf(amax, kept ? v * old : v);
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWriteThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  const int e = scale_exponent(amax);
  const float inv = pow2(-e);
  for (int x = threadIdx.x; x < total; x += kWriteThreads) {
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

// A thread per N codes of a row: N values of type T out (N = 16: one 16-byte load; N = 1: any head dim and alignment).
template <typename T, int N>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_wait();
  const int b = blockIdx.y, kv = blockIdx.z;
  int start, rows;
  if (!read_range(p, b, start, rows) && blockIdx.x == 0 && threadIdx.x == 0) report(p.status, TS_ERR_DEVICE_CHECK);
  const int per = p.d / N, heads = p.Hkv * per;
  const long long total = static_cast<long long>(p.n) * heads;
  const long long step = static_cast<long long>(gridDim.x) * kReadThreads;
  T* out = static_cast<T*>(p.out[kv]) + static_cast<long long>(b) * total * N;
  for (long long x = static_cast<long long>(blockIdx.x) * kReadThreads + threadIdx.x; x < total; x += step) {
    const int t = static_cast<int>(x / heads);
    const int rest = static_cast<int>(x - static_cast<long long>(t) * heads), h = rest / per, c = rest - h * per;
    float s = 0.f;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (t < rows) {
      const int pos = start + t, lp = pos / p.bs, row = pos - lp * p.bs;
      const int page = p.table[static_cast<long long>(b) * p.max_blocks + lp];
      if (page < 0 || page >= p.num_blocks) {
        report(p.status, TS_ERR_DEVICE_CHECK);
      } else {
        const long long head = static_cast<long long>(page) * p.Hkv + h;
        const uint8_t* from = p.cache[kv] + (head * p.bs + row) * p.d + c * N;
        s = scale_in_range(p.scale[kv][head * (p.bs / p.sb) + row / p.sb]);
        if constexpr (N == 16) w = *reinterpret_cast<const uint4*>(from);
        else w.x = *from;
      }
    }
    if constexpr (N == 1) {
      const float v = decode_e4m3(w.x) * s;
      if constexpr (sizeof(T) == 2) out[x] = __float2bfloat16_rn(v);
      else out[x] = v;
    } else {
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
      float v[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 lo = decode_e4m3x2(in[j]), hi = decode_e4m3x2(in[j] >> 16);
        v[4 * j] = lo.x * s, v[4 * j + 1] = lo.y * s, v[4 * j + 2] = hi.x * s, v[4 * j + 3] = hi.y * s;
      }
      if constexpr (sizeof(T) == 2) {
        uint4* to = reinterpret_cast<uint4*>(out + x * 16);
        to[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        to[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                           pack_bf16x2(v[14], v[15]));
      } else {
        float4* to = reinterpret_cast<float4*>(out + x * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
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
  c.n_keep = bad ? 0 : (c.L + c.a + p.bs - 1) / p.bs;
  c.p0 = bad ? 0 : c.L / p.bs;
  bad = bad || c.n_used - c.p0 > kMaxPages;
  if (!bad) {
    for (int j = threadIdx.x; j < c.a; j += blockDim.x) {
      const int32_t* path = p.accept_path + static_cast<long long>(b) * p.m;
      const int pj = path[j];
      s_path[j] = pj;
      if (j == 0 ? pj != 0 : (pj >= p.m || pj <= path[j - 1])) bad = true;
    }
    for (int i = c.p0 + threadIdx.x; i < c.n_used; i += blockDim.x) {
      const int pg = p.table[static_cast<long long>(b) * p.max_blocks + i];
      s_page[i - c.p0] = pg;
      if (pg < 0 || pg >= p.num_blocks) bad = true;
    }
  }
  c.ok = !__syncthreads_or(bad);
  return c;
}

// A CTA per (sequence, KV head, K or V).  The accepted rows' codes and scales are staged in shared memory, so every row is
// read before any is written; then a warp per block quantises its kept and its new rows.
template <int N>  // codes a load: 16, 4 or 1
__global__ void __launch_bounds__(kCommitThreads) commit_rows_kernel(const __grid_constant__ CommitParams p) {
  extern __shared__ __align__(16) unsigned char s_rows[];
  __shared__ int s_path[TS_MAX_NODES];
  __shared__ int s_page[kMaxPages];
  __shared__ float s_scale[TS_MAX_NODES];
  using Word = typename std::conditional<N == 16, uint4, typename std::conditional<N == 4, uint32_t, uint8_t>::type>::type;
  pdl_wait();
  const int b = blockIdx.y, h = blockIdx.x >> 1, kv = blockIdx.x & 1;
  const Commit c = commit_of(p, b, s_path, s_page);
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
  for (int blk = c.L / p.sb + warp; blk <= (c.L + c.a - 1) / p.sb; blk += kCommitThreads / 32) {
    const int first = blk * p.sb, kept = max(0, c.L - first), end = min(p.sb, c.L + c.a - first);
    uint8_t* codes = cache + (head_of(max(first, c.L)) * p.bs + first % p.bs) * p.d;
    float* sc = scale + head_of(max(first, c.L)) * nsb + first % p.bs / p.sb;
    const float old = kept > 0 ? scale_in_range(*sc) : 1.f;
    auto word = [&](int x) {
      const int r = x / per;
      return r < kept ? reinterpret_cast<const Word*>(codes)[x]
                      : reinterpret_cast<const Word*>(s_rows)[(first + r - c.L) * per + (x - r * per)];
    };
    auto by = [&](int x) {
      const int r = x / per;
      return r < kept ? old : s_scale[first + r - c.L];
    };
    float amax = 0.f;
    for (int x = lane; x < end * per; x += 32) {
      const Word w = word(x);
      const uint8_t* one = reinterpret_cast<const uint8_t*>(&w);
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) big = fmaxf(big, fabsf(decode_e4m3(one[j])));
      amax = fmaxf(amax, big * by(x));
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    const int e = scale_exponent(amax);
    for (int x = lane; x < end * per; x += 32) {
      Word w = word(x);
      const float f = by(x) * pow2(-e);
      uint8_t* one = reinterpret_cast<uint8_t*>(&w);
#pragma unroll
      for (int j = 0; j < N; ++j) one[j] = static_cast<uint8_t>(encode_e4m3x2(decode_e4m3(one[j]) * f, 0.f) & 0xFFu);
      reinterpret_cast<Word*>(codes)[x] = w;
    }
    __syncwarp();
    if (lane == 0) *sc = pow2(e);
  }
}

// Tables, lengths and the released pages, after the rows have moved: a CTA per sequence.
__global__ void __launch_bounds__(kCommitThreads) commit_table_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int s_path[TS_MAX_NODES];
  __shared__ int s_page[kMaxPages];
  pdl_wait();
  const int b = blockIdx.x;
  const Commit c = commit_of(p, b, s_path, s_page);
  const long long o = static_cast<long long>(b) * p.max_blocks;
  for (int i = threadIdx.x; i < p.max_blocks; i += kCommitThreads) {
    const int k = i + c.n_keep;
    p.freed[o + i] = c.ok && k < c.n_used ? s_page[k - c.p0] : -1;
    const bool gone = c.ok && i >= c.n_keep && i < c.n_used;
    if (gone) p.table_out[o + i] = -1;
    else if (p.table_out != p.table) p.table_out[o + i] = p.table[o + i];
  }
  if (threadIdx.x == 0) {
    p.freed_count[b] = c.ok ? c.n_used - c.n_keep : 0;
    p.prefix_out[b] = c.ok ? c.L + c.a : c.L;
    if (!c.ok) report(p.status, TS_ERR_DEVICE_CHECK);
  }
}

template <typename T>
cudaError_t launch_write(const WriteParams& p, bool wide, cudaStream_t stream) {
  const int chunks = (p.sb * p.d + kChunk - 1) / kChunk, held = 32 * kHeld;
  auto grid = [&](int w) { return dim3(static_cast<unsigned>((p.items + kWriteThreads / (32 * w) - 1) / (kWriteThreads / (32 * w)))); };
  const dim3 block(kWriteThreads);
  if (!wide) return launch_pdl(write_any_kernel<T>, dim3(static_cast<unsigned>(p.items)), block, 0, stream, p);
  if (chunks <= held) return launch_pdl(write_kernel<T, 1, true>, grid(1), block, 0, stream, p);
  if (chunks <= 2 * held) return launch_pdl(write_kernel<T, 2, true>, grid(2), block, 0, stream, p);
  if (chunks <= 4 * held) return launch_pdl(write_kernel<T, 4, true>, grid(4), block, 0, stream, p);
  if (chunks <= 8 * held) return launch_pdl(write_kernel<T, 8, true>, grid(8), block, 0, stream, p);
  return launch_pdl(write_kernel<T, 8, false>, grid(8), block, 0, stream, p);
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
  p.max_blocks = c.max_blocks, p.num_blocks = c.num_blocks;
  p.blocks = static_cast<int>((static_cast<long long>(c.n) + 2LL * c.scale_block - 2) / c.scale_block);
  p.items = 2LL * c.B * p.blocks * c.Hkv;
  if (p.items > INT32_MAX) return TS_ERR_UNSUPPORTED;
  const size_t size = c.dt == TS_BF16 ? 2 : 4;
  bool wide = c.d % kChunk == 0;
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
  const long long most = (16LL * num_sms + 2LL * c.B - 1) / (2LL * c.B);
  const unsigned gx = static_cast<unsigned>(std::max(1LL, std::min((total + kReadThreads - 1) / kReadThreads, std::max(1LL, most))));
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
  const uintptr_t at = reinterpret_cast<uintptr_t>(c.k_cache) | reinterpret_cast<uintptr_t>(c.v_cache) | static_cast<uintptr_t>(c.d);
  const size_t smem = static_cast<size_t>(c.m) * c.d;  // at most 64 KB
  auto run = [&](auto kernel, std::atomic<uint64_t>& done) {
    cudaError_t e = once_per_device(done, [&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TS_MAX_NODES * 256);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(2 * c.Hkv, c.B), dim3(kCommitThreads), smem, stream, p);
  };
  static std::atomic<uint64_t> done16{0}, done4{0}, done1{0};
  cudaError_t e = at % 16 == 0 ? run(commit_rows_kernel<16>, done16)
                               : at % 4 == 0 ? run(commit_rows_kernel<4>, done4) : run(commit_rows_kernel<1>, done1);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  e = launch_pdl(commit_table_kernel, dim3(c.B), dim3(kCommitThreads), 0, stream, p);
  count_launches(2);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
