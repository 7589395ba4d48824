// ts_tree_attention_fp8, CUDA-core path: fp32 queries (any head dim <= 256, any page size) and the bf16 shapes that
// the tensor-core path (tree_attention_fp8_tc.cu) does not take.
//
// Mathematics: rows are (node, head of the KV head's group); per row the running maximum M and sum l of the softmax in
// the log2 domain over tiles of 64 keys, in fp32 throughout:
//   x_j = q . (code_j * ks_j) * scale * log2 e,   l = sum 2^(x_j - M),   O = sum 2^(x_j - M) * code_j * vs_j
// A tile's codes are decoded once into fp32 in shared memory and serve up to 32 rows (64 where d <= 64), which is what the split is for:
// decoding costs more than the products of one row.  A thread of the 16 x 16 holds RPT rows x 4 keys of scores and RPT
// rows x 4 columns (per 64 of the head dim) of the output.  Long prefixes are cut into chunks, one CTA each, whose
// partial results a second kernel joins.
// Bound by the CUDA cores' issue slots and by shared memory (every product reads its operands there).
// Measured (GB300): fp32, 2 sequences of up to 700 tokens, 8 nodes, 8 heads on 2, d = 64: 16.7 us, the latency of one tile a chunk and of
// the join.  8 sequences of 4096 tokens, 8 heads on 2: 32 nodes at d = 64 119 us, one at d = 128 58 (its tiles take the shared memory
// 9000 cycles each, two thirds of the time, for four rows as for sixteen).  bf16 with d = 64, 32 heads on 8: 8 single tokens over 4096
// 138 us, 4 x 64 nodes over 4096 444, 27 and 99 times their floors.
#include <algorithm>

#include "fp8_cache.cuh"
#include "internal.h"

namespace ts {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 64;
constexpr int kMinTiles = 1;     // tiles that a chunk is worth
constexpr float kLn2f = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634074f;
// The least maximum of a row that has met a key.  A score below fp32's range, -inf, weighs nothing beside others; where there are no
// others the sum stays 0 under this maximum, and under -inf in a row without keys.
constexpr float kLeast = -3.402823466e38f;
constexpr uint32_t kMasked = 0x80000000u;  // weight -0: a key that the row does not attend to (its V may be NaN)

struct Params {
  const void* q;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* prefix_len;
  const uint64_t* mask;
  void* out;
  float* lse;
  float* part_o;    // [B * Hkv * rows, chunks, d]
  float2* part_ml;  // [B * Hkv * rows, chunks]: maximum (log2 units), sum
  int32_t* status;
  int B, m, Hq, Hkv, g, rows, d, dp, W, bs, sb, max_blocks, num_blocks, max_prefix, chunks, row_tiles;
  float scale_log2;
  bool wide;        // 16 codes a load
};

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A row's sum: NaN where it is 0 although the row has met a key (M: its maximum).
__device__ __forceinline__ float sum_of(float M, float l) { return l == 0.f && M != -INFINITY ? __int_as_float(0x7FC00000) : l; }

__device__ __forceinline__ bool usable(const Params& p, int L) {
  return L >= 0 && L <= p.max_prefix && static_cast<long long>(L) + p.m <= static_cast<long long>(p.max_blocks) * p.bs;
}

// What a tile's keys are: whether there is one, its place in the cache (in rows) and its scales.
struct Keys {
  int page[kKeys];  // -1: behind the end, or in a page without an id
  long long at[kKeys];
  float ks[kKeys], vs[kKeys];
};

// Sixteen codes times f -> s (16-byte aligned).
__device__ __forceinline__ void put16(float* s, const uint4& w, float f) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float2 lo = decode_e4m3x2(in[u]), hi = decode_e4m3x2(in[u] >> 16);
    *reinterpret_cast<float4*>(s + 4 * u) = make_float4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
  }
}
// The tile's values of one tensor -> s[64][pitch], code by code (zeros where there is no key and in the columns from d to dp).
__device__ void stage(const Params& p, const uint8_t* cache, const Keys& k, const float* scale, float* s, int pitch) {
  for (int x = threadIdx.x; x < kKeys * p.dp; x += kThreads) {
    const int j = x / p.dp, c = x - j * p.dp;
    s[j * pitch + c] = k.page[j] >= 0 && c < p.d ? decode_e4m3(cache[k.at[j] * p.d + c]) * scale[j] : 0.f;
  }
}

// RPT rows per thread (16 * RPT a CTA), CG groups of 64 head-dim columns.
template <typename T, int RPT, int CG>
__global__ void __launch_bounds__(kThreads) attn_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int ROWS = 16 * RPT;
  const int kp = p.dp + 4;                 // pitch of K rows: a half-warp reads 16 rows at one column
  float* sq = smem;                        // [ROWS][dp]
  float* sk = sq + ROWS * p.dp;            // [64][dp + 4]
  float* sv = sk + kKeys * kp;             // [64][dp]
  float* sp = sv + kKeys * p.dp;           // [ROWS][64]
  __shared__ Keys s_keys[2];
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y / p.row_tiles, R0 = (blockIdx.y % p.row_tiles) * ROWS, chunk = blockIdx.x;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int L = p.prefix_len[b];
  if (!usable(p, L)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(p.status, TS_ERR_DEVICE_CHECK);
    return;  // (the joining kernel passes over such a sequence)
  }
  const int nkeys = L + p.m, tiles = (nkeys + kKeys - 1) / kKeys;
  const int t0 = static_cast<int>(static_cast<long long>(chunk) * tiles / p.chunks);
  const int t1 = static_cast<int>(static_cast<long long>(chunk + 1) * tiles / p.chunks);
  const T* q = static_cast<const T*>(p.q);
  auto q_at = [&](int row) {  // offset of a row's query and output
    const int node = row / p.g, head = h * p.g + row % p.g;
    return (static_cast<long long>(b) * p.m + node) * p.Hq + head;
  };
  for (int x = threadIdx.x; x < ROWS * p.dp; x += kThreads) {
    const int r = x / p.dp, c = x - r * p.dp;
    sq[x] = R0 + r < p.rows && c < p.d ? load1(q + q_at(R0 + r) * p.d + c) : 0.f;
  }
  float M[RPT], l[RPT];
  float4 acc[RPT][CG];
  const uint64_t* words[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    M[r] = -INFINITY;
    l[r] = 0.f;
    const int row = min(R0 + ty * RPT + r, p.rows - 1);
    words[r] = p.mask + (static_cast<long long>(b) * p.m + row / p.g) * p.W;
#pragma unroll
    for (int c = 0; c < CG; ++c) acc[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // The first 64 threads look the keys up, a page's id three tiles ahead, its scales two; all of them ask for the codes of the next
  // tile while they compute this one.
  const int nsb = p.bs / p.sb;
  auto id_of = [&](int t) {
    const int pos = t * kKeys + static_cast<int>(threadIdx.x);
    return t < t1 && pos < nkeys ? max(-1, p.table[static_cast<long long>(b) * p.max_blocks + pos / p.bs]) : -2;
  };
  int id = -2, page = -1;  // of the tile after next; of the next
  long long at = 0;
  float ks = 0.f, vs = 0.f;
  auto look = [&](int t) {  // (id: that of tile t)
    page = -1, at = 0, ks = vs = 0.f;
    if (id == -2) return;
    if (id < 0 || id >= p.num_blocks) {
      report(p.status, TS_ERR_DEVICE_CHECK);
      return;
    }
    const int row = (t * kKeys + static_cast<int>(threadIdx.x)) % p.bs;
    const long long head = static_cast<long long>(id) * p.Hkv + h, block = head * nsb + row / p.sb;
    page = id, at = head * p.bs + row, ks = scale_in_range(p.ks[block]), vs = scale_in_range(p.vs[block]);
  };
  auto keep = [&](int t) {
    Keys& k = s_keys[t & 1];
    k.page[threadIdx.x] = page, k.at[threadIdx.x] = at, k.ks[threadIdx.x] = ks, k.vs[threadIdx.x] = vs;
  };
  const bool finder = threadIdx.x < kKeys;
  const int per = p.d / 16;
  uint4 kc[CG], vc[CG];
  auto ask = [&](int t) {
    const Keys& k = s_keys[t & 1];
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      const int x = threadIdx.x + kThreads * i, j = x / per;
      kc[i] = vc[i] = make_uint4(0, 0, 0, 0);
      if (j < kKeys && k.page[j] >= 0) {
        const long long o = k.at[j] * p.d + (x - j * per) * 16;
        kc[i] = *reinterpret_cast<const uint4*>(p.kc + o);
        vc[i] = *reinterpret_cast<const uint4*>(p.vc + o);
      }
    }
  };
  if (finder) {
    id = id_of(t0);
    look(t0);
    keep(t0);
    id = id_of(t0 + 1);
    look(t0 + 1);
    id = id_of(t0 + 2);
  }
  __syncthreads();
  if (p.wide) ask(t0);
  for (int t = t0; t < t1; ++t) {
    const int key0 = t * kKeys;
    const Keys& keys = s_keys[t & 1];
    const int* s_page = keys.page;
    if (p.wide) {
#pragma unroll
      for (int i = 0; i < CG; ++i) {
        const int x = threadIdx.x + kThreads * i, j = x / per, c = (x - j * per) * 16;
        if (j < kKeys) {
          put16(sk + j * kp + c, kc[i], keys.ks[j]);
          put16(sv + j * p.dp + c, vc[i], keys.vs[j]);
        }
      }
    } else {
      stage(p, p.kc, keys, keys.ks, sk, kp);
      stage(p, p.vc, keys, keys.vs, sv, p.dp);
    }
    if (finder) {
      keep(t + 1);
      look(t + 2);
      id = id_of(t + 3);
    }
    __syncthreads();
    if (p.wide) ask(t + 1);
    float x[RPT][4];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[r][j] = 0.f;
    for (int c = 0; c < p.dp; c += 4) {
      float4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * kp + c);
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float4 a = *reinterpret_cast<const float4*>(sq + (ty * RPT + r) * p.dp + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[r][j] = fmaf(a.x, kk[j].x, fmaf(a.y, kk[j].y, fmaf(a.z, kk[j].z, fmaf(a.w, kk[j].w, x[r][j]))));
      }
    }
    bool hidden = false;  // whether any key of the tile is left out for some row
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      bool seen[4], any = false;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pos = key0 + tx + 16 * j, n = pos - L;
        seen[j] = s_page[tx + 16 * j] >= 0 && (n < 0 || ((words[r][n >> 6] >> (n & 63)) & 1ull));
        any = any || seen[j];
        x[r][j] *= p.scale_log2;
        if (seen[j]) top = fmaxf(top, x[r][j]);
      }
      if (any) top = fmaxf(top, kLeast);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float M2 = fmaxf(M[r], top);
      const float keep = M[r] == M2 ? 1.f : exp2f(M[r] - M2);  // (equal infinities too)
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (a NaN score gives a NaN weight; the maximum passed over it)
        const float w = seen[j] ? (x[r][j] == -INFINITY ? 0.f : exp2f(x[r][j] - M2)) : __uint_as_float(kMasked);
        if (seen[j]) sum += w;
        sp[(ty * RPT + r) * kKeys + tx + 16 * j] = w;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[r] = l[r] * keep + sum;
      M[r] = M2;
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        acc[r][c].x *= keep, acc[r][c].y *= keep, acc[r][c].z *= keep, acc[r][c].w *= keep;
      }
    }
    hidden = key0 + kKeys > L;
#pragma unroll
    for (int j = 0; j < 4; ++j) hidden = hidden || s_page[tx + 16 * j] < 0;
    hidden = __any_sync(0xffffffffu, hidden);
    __syncwarp();  // (a row's weights are written and read by one half-warp)
    for (int j = 0; j < kKeys; ++j) {
      float w[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) w[r] = sp[(ty * RPT + r) * kKeys + j];
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        const int col = 4 * tx + 64 * c;
        if (col < p.dp) {
          const float4 v = *reinterpret_cast<const float4*>(sv + j * p.dp + col);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            if (hidden && __float_as_uint(w[r]) == kMasked) continue;
            acc[r][c].x = fmaf(w[r], v.x, acc[r][c].x);
            acc[r][c].y = fmaf(w[r], v.y, acc[r][c].y);
            acc[r][c].z = fmaf(w[r], v.z, acc[r][c].z);
            acc[r][c].w = fmaf(w[r], v.w, acc[r][c].w);
          }
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = R0 + ty * RPT + r;
    if (row >= p.rows) continue;
    const bool whole = p.chunks == 1;
    const float sum = whole ? sum_of(M[r], l[r]) : l[r], inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long unit = (static_cast<long long>(b) * p.Hkv + h) * p.rows + row;
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      const float v[4] = {acc[r][c].x, acc[r][c].y, acc[r][c].z, acc[r][c].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = 4 * tx + 64 * c + u;
        if (col >= p.d) continue;
        if (whole) store1(static_cast<T*>(p.out) + q_at(row) * p.d + col, v[u] * inv);
        else p.part_o[(unit * p.chunks + chunk) * p.d + col] = v[u];
      }
    }
    if (tx == 0) {
      if (!whole) p.part_ml[unit * p.chunks + chunk] = make_float2(M[r], l[r]);
      else if (p.lse != nullptr) p.lse[q_at(row)] = sum == 0.f ? -INFINITY : (M[r] + log2f(sum)) * kLn2f;
    }
  }
}

// A CTA per row: its warps take the chunks in turn, four of them in flight each, and their sums are joined in the warps' order.  (A warp
// per row, a chunk after the other, waited for each: 20 of 74 us for 8 single tokens of 8 heads over 4096 tokens.)
constexpr int kJoinWarps = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params p) {
  __shared__ float s_acc[kJoinWarps][256], s_l[kJoinWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = blockIdx.x;
  const int bh = static_cast<int>(blockIdx.x) / p.rows, row = static_cast<int>(blockIdx.x) - bh * p.rows, b = bh / p.Hkv, h = bh - b * p.Hkv;
  if (!usable(p, p.prefix_len[b])) return;
  const float2* ml = p.part_ml + unit * p.chunks;
  const float* part = p.part_o + unit * p.chunks * p.d;
  float M = -INFINITY;
  for (int c = lane; c < p.chunks; c += 32) M = fmaxf(M, ml[c].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float l = 0.f, acc[8] = {};
#pragma unroll 4
  for (int c = warp; c < p.chunks; c += kJoinWarps) {
    const float2 x = ml[c];
    const float f = x.y == 0.f ? 0.f : x.x == M ? 1.f : exp2f(x.x - M);  // (0: no key in that chunk; a NaN sum goes on)
    l = fmaf(x.y, f, l);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int col = lane + 32 * u;
      if (col < p.d) acc[u] = fmaf(part[static_cast<long long>(c) * p.d + col], f, acc[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) s_acc[warp][lane + 32 * u] = acc[u];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = s_l[0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) l += s_l[w];
  l = sum_of(M, l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int node = row / p.g, head = h * p.g + row - node * p.g;
  const long long o = (static_cast<long long>(b) * p.m + node) * p.Hq + head;
  for (int col = threadIdx.x; col < p.d; col += 32 * kJoinWarps) {
    float v = s_acc[0][col];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) v += s_acc[w][col];
    store1(static_cast<T*>(p.out) + o * p.d + col, v * inv);
  }
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[o] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2f;
}

// Rows per CTA: 16 where there are no more, 32 otherwise (the decoded tile serves them all).  64 halve what a row reads of the shared
// memory: 128 rows of 4096 tokens, d = 64, 166 -> 121 us; at d = 128 they leave one CTA an SM (224 rows 130 -> 174, not taken).
int rows_per_cta(int rows, int d) { return rows <= 16 ? 16 : rows <= 32 || d > 64 ? 32 : 64; }

// Chunks per (sequence, KV head, row tile): two CTAs per SM's worth, of kMinTiles tiles at least.
int chunks_of(int B, int m, int Hq, int Hkv, int d, int max_prefix, int num_sms) {
  const long long rows = static_cast<long long>(m) * (Hq / Hkv);
  const long long tiles = (static_cast<long long>(max_prefix) + m + kKeys - 1) / kKeys;
  const long long units = static_cast<long long>(B) * Hkv * ((rows + rows_per_cta(static_cast<int>(rows), d) - 1) / rows_per_cta(static_cast<int>(rows), d));
  const long long want = std::max(1LL, 2LL * num_sms / units);
  return static_cast<int>(std::max(1LL, std::min(want, tiles / kMinTiles)));
}

template <typename T, int RPT, int CG>
cudaError_t launch_attn(const Params& p, dim3 grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int most = (16 * RPT * 64 * CG + kKeys * (64 * CG + 4) + kKeys * 64 * CG + 16 * RPT * kKeys) * 4;
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attn_kernel<T, RPT, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  const size_t smem = (16 * RPT * p.dp + kKeys * (p.dp + 4) + kKeys * p.dp + 16 * RPT * kKeys) * sizeof(float);
  return launch_pdl(attn_kernel<T, RPT, CG>, grid, dim3(kThreads), smem, stream, p);
}
template <typename T, int RPT>
cudaError_t launch_attn_cg(const Params& p, dim3 grid, cudaStream_t stream) {
  switch ((p.dp + 63) / 64) {
    case 1: return launch_attn<T, RPT, 1>(p, grid, stream);
    case 2: return launch_attn<T, RPT, 2>(p, grid, stream);
    case 3: return launch_attn<T, RPT, 3>(p, grid, stream);
    default: return launch_attn<T, RPT, 4>(p, grid, stream);
  }
}
template <typename T>
cudaError_t launch_all(const Params& p, cudaStream_t stream) {
  const dim3 grid(p.chunks, p.Hkv * p.row_tiles, p.B);
  cudaError_t e;
  switch (rows_per_cta(p.rows, p.d)) {
    case 16: e = launch_attn_cg<T, 1>(p, grid, stream); break;
    case 32: e = launch_attn_cg<T, 2>(p, grid, stream); break;
    default: e = launch_attn<T, 4, 1>(p, grid, stream); break;
  }
  if (e != cudaSuccess || p.chunks == 1) return e;
  return launch_pdl(join_kernel<T>, dim3(static_cast<unsigned>(p.B * p.Hkv * p.rows)), dim3(32 * kJoinWarps), 0, stream, p);
}

}  // namespace

size_t attention_fp8_simt_workspace_bytes(int B, int m, int Hq, int Hkv, int d, int max_prefix, int num_sms) {
  const int chunks = chunks_of(B, m, Hq, Hkv, d, max_prefix, std::max(1, num_sms));
  if (chunks == 1) return 256;
  return static_cast<size_t>(B) * m * Hq * chunks * (static_cast<size_t>(d) * 4 + 8) + 256;
}

int attention_fp8_simt_launch(const Fp8AttnCall& a, cudaStream_t stream, int num_sms) {
  Params p;
  p.q = a.q;
  p.kc = static_cast<const uint8_t*>(a.k_cache), p.vc = static_cast<const uint8_t*>(a.v_cache);
  p.ks = a.k_scale, p.vs = a.v_scale;
  p.table = a.block_table, p.prefix_len = a.prefix_len, p.mask = a.mask, p.out = a.out, p.lse = a.lse, p.status = a.dev_status;
  p.B = a.B, p.m = a.m, p.Hq = a.Hq, p.Hkv = a.Hkv, p.g = a.Hq / a.Hkv, p.rows = a.m * p.g, p.d = a.d, p.dp = (a.d + 3) / 4 * 4;
  p.W = (a.m + 63) / 64, p.bs = a.block_size, p.sb = a.scale_block, p.max_blocks = a.max_blocks, p.num_blocks = a.num_blocks;
  p.max_prefix = a.max_prefix;
  p.chunks = chunks_of(a.B, a.m, a.Hq, a.Hkv, a.d, a.max_prefix, num_sms);
  p.row_tiles = (p.rows + rows_per_cta(p.rows, p.d) - 1) / rows_per_cta(p.rows, p.d);
  if (static_cast<long long>(p.Hkv) * p.row_tiles > 65535) return TS_ERR_UNSUPPORTED;
  p.scale_log2 = a.scale * kLog2e;
  p.wide = a.d % 16 == 0 && (reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache)) % 16 == 0;
  const size_t rows = static_cast<size_t>(a.B) * a.m * a.Hq * p.chunks;  // (8-byte pairs first, then floats)
  p.part_ml = static_cast<float2*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + rows * sizeof(float2));
  const cudaError_t e = a.dt == TS_BF16 ? launch_all<__nv_bfloat16>(p, stream) : launch_all<float>(p, stream);
  count_launches(p.chunks == 1 ? 1 : 2);
  return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

}  // namespace ts
