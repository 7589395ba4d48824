// The page pool: ts_kv_reserve, ts_kv_fork, ts_kv_compact.
//
// State: a block table per sequence and refs, the number of table entries that name each page.
// What a call decides (which pages are free, who gets which, what moves where) is bookkeeping over
// refs and the tables: a few kilobytes to a few megabytes with a global order in it, so it is
// bound by latency.  reserve and compact run it as ONE thread-block cluster of eight CTAs: each CTA
// takes a contiguous share of the pages, and a step that needs everyone's result (how many free
// pages lie before mine) is a hardware cluster barrier, not another launch.  The rows of K and V
// that change place are then copied by a second, wide launch, bound by HBM.  fork has no global
// order (counts change by whole numbers, which commute) and runs wide from the start.
//
// Measured on the device (GB300, graph replays): reserve for 8 sequences of up to 8192 tokens 12.4 us, with the last
// pages of 256 fork rows copied (25 MB each way) 19-20 us; forks 6.3 us (one row to eight) and 8.3 us (512 rows);
// compact 10.6 us for 4 sequences, 147 us where some 6100 of 18400 pages in use move (64 KB of K and V each; the
// moves alone run at 6 TB/s).
//
// Free pages are always handed out in increasing id and requests are ranked by (sequence,
// logical page), by prefix sums, so the outcome does not depend on the order of execution.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace ts {
namespace {

constexpr int kPoolCtas = 8;        // one cluster (the portable limit)
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Exclusive prefix sum of v over the CTA's threads; *total is the sum.  Two barriers.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int w = s_warp[lane];  // kPoolWarps == 32: every warp sums the warps' totals for itself
  int winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += y;
  }
  const int before = __shfl_sync(0xffffffffu, winc - w, warp);
  *total = __shfl_sync(0xffffffffu, winc, 31);
  __syncthreads();
  return before + inc - v;
}

// One value per CTA of the cluster: everyone gets the sum of the lower ranks' and the total.
// Contains a cluster barrier (also for the global memory written before it).
__device__ __forceinline__ int cluster_scan(int mine, int* s_all, int* total) {
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x < kPoolCtas) st_dsmem_u32(dsmem_addr(smem_u32(s_all + rank), threadIdx.x), mine);
  cluster_sync_all();
  int before = 0, sum = 0;
#pragma unroll
  for (int c = 0; c < kPoolCtas; ++c) {
    before += c < static_cast<int>(rank) ? s_all[c] : 0;
    sum += s_all[c];
  }
  *total = sum;
  return before;
}

// ------------------------------------------------------------------------------------ reserve
struct ReserveArgs {
  const int32_t* table;
  const int32_t* prefix_len;
  const int32_t* refs;
  const int32_t* freed;
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* granted;
  int32_t* copy;       // [B, 2] page to copy from and to (from -1: none)
  int32_t* free_list;  // the lowest free pages, as many as are asked for
  int32_t* status;
  long long n;
  int num_blocks, bs, max_blocks, B, num_freed;
};

// The row's logical pages [first, last) for positions L .. L+n-1; false for a bad state.
__device__ __forceinline__ bool row_span(const ReserveArgs& a, int b, int* L, int* first, int* last) {
  *L = a.prefix_len[b];
  if (*L < 0 || *L + a.n > static_cast<long long>(a.max_blocks) * a.bs) return false;
  *first = *L / a.bs;
  *last = static_cast<int>((*L + a.n + a.bs - 1) / a.bs);
  return true;
}

// Steps, with a cluster barrier between each two: copy the state; release; count what each row lacks and the free
// pages of each CTA's share; (where last pages are shared) decide who copies; number the requests and list the
// lowest free pages; hand them out.  What all CTAs need to know of a row (its shared last page, how many pages
// it wants) is written straight into every CTA's shared memory; what only its own warp needs stays in registers
// (lane k of a warp holds that of its k-th row).  A step costs its dependent loads, some 1300 cycles each.
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1) reserve_kernel(const ReserveArgs a) {
  __shared__ int s_warp[32], s_all[2][kPoolCtas], s_first_short, s_shared;
  __shared__ int s_want[TS_MAX_POOL_ROWS], s_tail[TS_MAX_POOL_ROWS];
  constexpr int RUN = 4 * kPoolThreads;  // pages of a share looked at at a time, four neighbours per thread
  const int rank = static_cast<int>(cluster_ctarank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = rank * kPoolThreads + tid, gthreads = kPoolCtas * kPoolThreads;
  const int gwarp = rank * kPoolWarps + warp, gwarps = kPoolCtas * kPoolWarps;
  if (tid == 0) {
    s_first_short = a.B;
    s_shared = 0;
  }
  pdl_wait();
  // the new state starts as the old one
  if (a.refs_out != a.refs)
    for (int i = gtid; i < a.num_blocks; i += gthreads) a.refs_out[i] = a.refs[i];
  if (a.table_out != a.table) {
    const long long cells = static_cast<long long>(a.B) * a.max_blocks;
    for (long long i = gtid; i < cells; i += gthreads) a.table_out[i] = a.table[i];
  }
  cluster_sync_all();  // (also: every CTA runs before its shared memory is written to)
  const int32_t* refs = a.refs;
  if (a.num_freed > 0) {
    for (int i = gtid; i < a.num_freed; i += gthreads) {
      const int p = a.freed[i];
      if (p < 0) continue;
      if (p >= a.num_blocks) {
        report(a.status, TS_ERR_DEVICE_CHECK);
      } else if (atomicSub(a.refs_out + p, 1) <= 0) {  // undone: the sum is the same in every order
        atomicAdd(a.refs_out + p, 1);
        report(a.status, TS_ERR_DEVICE_CHECK);
      }
    }
    refs = a.refs_out;
    cluster_sync_all();
  }
  // free pages of this CTA's share (a bit per page; the first run's stay in a register)
  const int share = (a.num_blocks + kPoolCtas * RUN - 1) / (kPoolCtas * RUN) * RUN;
  const int lo = static_cast<int>(min(static_cast<long long>(rank) * share, static_cast<long long>(a.num_blocks)));
  const int hi = min(lo + share, a.num_blocks);
  auto free_bits = [&](int i0) -> unsigned {
    unsigned bits = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + 4 * tid + u < hi && __ldcg(refs + i0 + 4 * tid + u) == 0) bits |= 1u << u;
    return bits;
  };
  const unsigned first_run = free_bits(lo);
  // what each row lacks, and whether its last page is shared; a warp per row
  int my_want = 0, my_refs = 0;
  bool my_copy = false;
  for (int b = gwarp, k = 0; b < a.B; b += gwarps, ++k) {
    int L, first, last, need = 0, tail = -1, tail_refs = 0;
    bool ok = row_span(a, b, &L, &first, &last);
    if (ok) {
      const int32_t* row = a.table + static_cast<long long>(b) * a.max_blocks;
      bool bad = false;
      for (int i0 = first; i0 < last; i0 += 32) {
        const int p = i0 + lane < last ? row[i0 + lane] : 0;
        bad |= p < -1 || p >= a.num_blocks;
        need += __popc(__ballot_sync(0xffffffffu, i0 + lane < last && p == -1));
        if (i0 == first) tail = __shfl_sync(0xffffffffu, p, 0);
      }
      ok = !__any_sync(0xffffffffu, bad);
      if (L % a.bs == 0 || !ok) tail = -1;
      if (tail >= 0) tail_refs = __ldcg(refs + tail);
      if (tail_refs <= 1) tail = -1;
    }
    if (!ok && lane == 0) report(a.status, TS_ERR_DEVICE_CHECK);
    if (lane < kPoolCtas) {
      st_dsmem_u32(dsmem_addr(smem_u32(s_want + b), lane), ok ? need : -1);
      st_dsmem_u32(dsmem_addr(smem_u32(s_tail + b), lane), tail);
    }
    if (tail >= 0 && lane == 0) atomicAdd(&s_shared, 1);
    if (lane == k) {
      my_want = ok ? need : -1;
      my_refs = tail_refs;
    }
  }
  int nfree = 0, here;
  for (int i0 = lo; i0 < hi; i0 += RUN) nfree += __popc(i0 == lo ? first_run : free_bits(i0));
  block_scan(nfree, s_warp, &here);
  if (tid < kPoolCtas) {
    st_dsmem_u32(dsmem_addr(smem_u32(&s_all[0][rank]), tid), here);
    st_dsmem_u32(dsmem_addr(smem_u32(&s_all[1][rank]), tid), s_shared);
  }
  cluster_sync_all();
  int F = 0, free_before = 0, any_shared = 0;
#pragma unroll
  for (int c = 0; c < kPoolCtas; ++c) {
    free_before += c < rank ? s_all[0][c] : 0;
    F += s_all[0][c];
    any_shared += s_all[1][c];
  }
  // of the rows that share a last page, each copies it as long as another reference is left
  for (int b = gwarp, k = 0; b < a.B; b += gwarps, ++k) {
    const int t = s_tail[b];
    bool copies = false;
    if (t >= 0) {
      int before = 0;
      for (int j = lane; j < b; j += 32) before += s_tail[j] == t;
      before = __reduce_add_sync(0xffffffffu, before);
      copies = __shfl_sync(0xffffffffu, my_refs, k) - before > 1;
      if (lane == k) {
        my_copy = copies;
        my_want += copies;
      }
      const int w = __shfl_sync(0xffffffffu, my_want, k);
      if (copies && lane < kPoolCtas) st_dsmem_u32(dsmem_addr(smem_u32(s_want + b), lane), w);
    }
    if (lane < 2) a.copy[2 * b + lane] = lane == 0 && copies ? t : -1;
  }
  if (any_shared > 0) cluster_sync_all();
  else __syncthreads();
  // where each row's requests start in the order (every CTA for itself), in place of how many they are
  int R = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPoolThreads) {
    const int w = b0 + tid < a.B ? max(0, s_want[b0 + tid]) : 0;
    int sum;
    const int at = block_scan(w, s_warp, &sum);
    if (b0 + tid < a.B) s_want[b0 + tid] = R + at;
    if (w > 0 && R + at + w > F) atomicMin(&s_first_short, b0 + tid);
    R += sum;
  }
  // this CTA's free pages that somebody gets
  int at = free_before;
  for (int i0 = lo; i0 < hi && at < R; i0 += RUN) {
    const unsigned bits = i0 == lo ? first_run : free_bits(i0);
    int sum;
    int r = at + block_scan(__popc(bits), s_warp, &sum);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if ((bits >> u) & 1u) {
        if (r < R) a.free_list[r] = i0 + 4 * tid + u;
        ++r;
      }
    }
    at += sum;
  }
  cluster_sync_all();
  const int first_short = s_first_short;
  for (int b = gwarp, k = 0; b < a.B; b += gwarps, ++k) {
    const int w = __shfl_sync(0xffffffffu, my_want, k);
    const bool copies = __shfl_sync(0xffffffffu, my_copy ? 1 : 0, k) != 0;
    bool is_short = w > 0 && b >= first_short;
    if (w == 0 && b > first_short && s_tail[b] >= 0) {
      // it was to keep its last page because others before it would have left it: not all have
      int left = 0;
      for (int j = lane; j < first_short; j += 32) left += s_tail[j] == s_tail[b];
      is_short = __shfl_sync(0xffffffffu, my_refs, k) - __reduce_add_sync(0xffffffffu, left) > 1;
    }
    if (w <= 0 || is_short) {
      if (lane == 0) {
        a.granted[b] = is_short ? -1 : w;
        if (copies) a.copy[2 * b] = -1;
        if (is_short) report(a.status, TS_ERR_NO_PAGES);
      }
      continue;
    }
    int L, first, last;
    row_span(a, b, &L, &first, &last);
    int32_t* row = a.table_out + static_cast<long long>(b) * a.max_blocks;
    int r = s_want[b];
    for (int i0 = first; i0 < last; i0 += 32) {
      const int i = i0 + lane;
      const bool take = i < last && ((i == first && copies) || __ldcg(row + i) == -1);
      const unsigned m = __ballot_sync(0xffffffffu, take);
      if (take) {
        const int page = __ldcg(a.free_list + r + __popc(m & ((1u << lane) - 1u)));
        row[i] = page;
        a.refs_out[page] = 1;
        if (i == first && copies) {
          a.copy[2 * b + 1] = page;
          atomicSub(a.refs_out + s_tail[b], 1);
        }
      }
      r += __popc(m);
    }
    if (lane == 0) a.granted[b] = w;
  }
}

// The scales of an 8-bit cache, nsb for every page and head; none: k is null.
struct Scales {
  float* k;
  float* v;
  int nsb;
};

// The first L % bs rows of the shared last pages, for every KV head: CTA (head, row b); with them the scales of the blocks
// that those rows reach.
template <typename Chunk>
__global__ void __launch_bounds__(256) copy_tails_kernel(unsigned char* kc, unsigned char* vc, int Hkv, int bs, int row_bytes,
                                                         Scales scales, const int32_t* __restrict__ copy,
                                                         const int32_t* __restrict__ prefix_len) {
  pdl_wait();
  const int b = blockIdx.y, h = blockIdx.x;
  const int from = copy[2 * b], to = copy[2 * b + 1];
  if (from < 0 || to < 0) return;
  const int rows = prefix_len[b] % bs, chunks = rows * (row_bytes / static_cast<int>(sizeof(Chunk)));
  if (scales.k != nullptr) {
    const int sb = bs / scales.nsb, blocks = rows > 0 ? (rows - 1) / sb + 1 : 0;
    const long long sf = (static_cast<long long>(from) * Hkv + h) * scales.nsb, st = (static_cast<long long>(to) * Hkv + h) * scales.nsb;
    for (int i = threadIdx.x; i < blocks; i += 256) {
      scales.k[st + i] = scales.k[sf + i];
      scales.v[st + i] = scales.v[sf + i];
    }
  }
  const long long page = static_cast<long long>(bs) * row_bytes;
  const long long src = (static_cast<long long>(from) * Hkv + h) * page, dst = (static_cast<long long>(to) * Hkv + h) * page;
  const Chunk* ks = reinterpret_cast<const Chunk*>(kc + src);
  const Chunk* vs = reinterpret_cast<const Chunk*>(vc + src);
  Chunk* kd = reinterpret_cast<Chunk*>(kc + dst);
  Chunk* vd = reinterpret_cast<Chunk*>(vc + dst);
  for (int i0 = threadIdx.x; i0 < chunks; i0 += 256 * 4) {
    Chunk k[4], v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 + 256 * u < chunks) {
        k[u] = ks[i0 + 256 * u];
        v[u] = vs[i0 + 256 * u];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 + 256 * u < chunks) {
        kd[i0 + 256 * u] = k[u];
        vd[i0 + 256 * u] = v[u];
      }
    }
  }
}

// --------------------------------------------------------------------------------------- fork
struct ForkArgs {
  const int32_t* table;
  const int32_t* prefix_len;
  const int32_t* refs;
  const int32_t* src;
  int32_t* table_out;
  int32_t* prefix_out;
  int32_t* refs_out;
  int32_t* status;
  int max_blocks, num_blocks, bs, B, B_out;
};
constexpr int kForkThreads = 256;

// New rows, and refs_out = refs where they are different buffers: the share of CTA `cta` of `ctas`.
__device__ __forceinline__ void fork_rows(const ForkArgs& a, int cta, int ctas) {
  const int tid = threadIdx.x, max_blocks = a.max_blocks, num_blocks = a.num_blocks, bs = a.bs, B = a.B, B_out = a.B_out;
  const int32_t *table = a.table, *prefix_len = a.prefix_len, *src = a.src;
  int32_t *table_out = a.table_out, *prefix_out = a.prefix_out, *status = a.status;
  for (int r = cta; r < B_out; r += ctas) {
    const int s = src[r];
    bool bad = s < -1 || s >= B;
    int L = 0;
    if (!bad && s >= 0) {
      L = prefix_len[s];
      if (L < 0 || L > static_cast<long long>(max_blocks) * bs) {
        bad = true;
        L = 0;
      }
    }
    const int kept = static_cast<int>((static_cast<long long>(L) + bs - 1) / bs);
    int32_t* row = table_out + static_cast<long long>(r) * max_blocks;
    for (int i = tid; i < max_blocks; i += 256) {
      int p = -1;
      if (i < kept) {
        p = table[static_cast<long long>(s) * max_blocks + i];
        if (p < 0 || p >= num_blocks) {
          p = -1;
          bad = true;
        }
      }
      row[i] = p;
    }
    if (bad) report(status, TS_ERR_DEVICE_CHECK);
    if (tid == 0) prefix_out[r] = L;
  }
  if (a.refs_out != a.refs)
    for (int i = cta * kForkThreads + tid; i < num_blocks; i += ctas * kForkThreads) a.refs_out[i] = a.refs[i];
}

// Counts: an entry of old row s among its kept pages is named once less and once more per new row
// that continues s; an entry beyond them is only let go.  Rows continued exactly once cost no
// atomic for their kept pages.
__device__ __forceinline__ void fork_refs(const ForkArgs& a, int cta, int ctas) {
  __shared__ int s_sum[8];
  const int tid = threadIdx.x, max_blocks = a.max_blocks, num_blocks = a.num_blocks, bs = a.bs, B = a.B, B_out = a.B_out;
  const int32_t *table = a.table, *prefix_len = a.prefix_len, *src = a.src;
  int32_t *refs_out = a.refs_out, *status = a.status;
  for (int s = cta; s < B; s += ctas) {
    int times = 0;
    for (int r = tid; r < B_out; r += 256) times += src[r] == s;
    times = __reduce_add_sync(0xffffffffu, times);
    __syncthreads();
    if ((tid & 31) == 0) s_sum[tid >> 5] = times;
    __syncthreads();
    times = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) times += s_sum[w];
    const int L = prefix_len[s];
    const bool bad = L < 0 || L > static_cast<long long>(max_blocks) * bs;
    const int kept = bad ? 0 : static_cast<int>((static_cast<long long>(L) + bs - 1) / bs);
    for (int i = tid; i < max_blocks; i += 256) {
      const int delta = (i < kept ? times : 0) - 1;
      if (delta == 0) continue;
      const int p = table[static_cast<long long>(s) * max_blocks + i];
      if (p == -1) continue;
      if (p < 0 || p >= num_blocks) {
        report(status, TS_ERR_DEVICE_CHECK);
      } else if (atomicAdd(refs_out + p, delta) + delta < 0) {
        report(status, TS_ERR_DEVICE_CHECK);
      }
    }
  }
}

__global__ void __launch_bounds__(kForkThreads) fork_rows_kernel(const ForkArgs a) {
  pdl_wait();
  fork_rows(a, blockIdx.x, gridDim.x);
}
__global__ void __launch_bounds__(kForkThreads) fork_refs_kernel(const ForkArgs a) {
  pdl_wait();
  fork_refs(a, blockIdx.x, gridDim.x);
}
// Both in one launch by one cluster, the barrier between them the cluster's.
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kForkThreads) fork_small_kernel(const ForkArgs a) {
  pdl_wait();
  fork_rows(a, blockIdx.x, kPoolCtas);
  cluster_sync_all();
  fork_refs(a, blockIdx.x, kPoolCtas);
}

// ------------------------------------------------------------------------------------ compact
struct CompactArgs {
  const int32_t* refs;
  int32_t* refs_out;
  int32_t* remap;
  int32_t* live;
  int32_t* moves;  // [0] how many, then (from, to) pairs
  int num_blocks;
};

// A CTA's share of the pages is cut into runs of 4096, four neighbouring pages per thread; the first run's counts
// stay in registers (pools of up to 32768 pages have no other), longer shares read theirs again.
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1) compact_kernel(const CompactArgs a) {
  __shared__ int s_warp[32], s_all[3][kPoolCtas];
  constexpr int RUN = 4 * kPoolThreads;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tid = threadIdx.x, gtid = rank * kPoolThreads + tid, gthreads = kPoolCtas * kPoolThreads;
  cluster_sync_all();  // every CTA of the cluster runs before its shared memory is written to
  pdl_wait();
  const int share = (a.num_blocks + kPoolCtas * RUN - 1) / (kPoolCtas * RUN) * RUN;
  const int lo = static_cast<int>(min(static_cast<long long>(rank) * share, static_cast<long long>(a.num_blocks)));
  const int hi = min(lo + share, a.num_blocks);
  int n0[4];
  auto load = [&](int i0, int (&n)[4]) {  // references of this thread's four pages of the run from i0 (0 past the share)
#pragma unroll
    for (int u = 0; u < 4; ++u) n[u] = i0 + 4 * tid + u < hi ? a.refs[i0 + 4 * tid + u] : 0;
  };
  load(lo, n0);
  int used = 0, sum;
  for (int i0 = lo; i0 < hi; i0 += RUN) {
    int n[4] = {n0[0], n0[1], n0[2], n0[3]};
    if (i0 > lo) load(i0, n);
#pragma unroll
    for (int u = 0; u < 4; ++u) used += n[u] > 0;
  }
  block_scan(used, s_warp, &sum);
  int live;
  cluster_scan(sum, s_all[0], &live);
  // free pages below `live` and pages in use from there on: as many of the one as of the other
  int holes = 0, movers = 0, hsum, msum;
  for (int i0 = lo; i0 < hi; i0 += RUN) {
    int n[4] = {n0[0], n0[1], n0[2], n0[3]};
    if (i0 > lo) load(i0, n);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 4 * tid + u;
      holes += i < hi && i < live && n[u] <= 0;
      movers += i >= live && n[u] > 0;
    }
  }
  block_scan(holes, s_warp, &hsum);
  block_scan(movers, s_warp, &msum);
  int htotal, mtotal;
  int hat = cluster_scan(hsum, s_all[1], &htotal);
  int mat = cluster_scan(msum, s_all[2], &mtotal);
  for (int i0 = lo; i0 < hi; i0 += RUN) {
    int n[4] = {n0[0], n0[1], n0[2], n0[3]};
    if (i0 > lo) load(i0, n);
    int kinds = 0;  // holes in the low half, movers in the high one
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 4 * tid + u;
      kinds += (i < hi && i < live && n[u] <= 0) + (static_cast<int>(i >= live && n[u] > 0) << 16);
    }
    int s;
    const int at = block_scan(kinds, s_warp, &s);
    int h = hat + (at & 0xffff), m = mat + (at >> 16);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 4 * tid + u;
      if (i >= hi) break;
      const bool use = n[u] > 0, hole = i < live && !use, mover = i >= live && use;
      if (hole) a.moves[2 + 2 * h++] = i;
      if (mover) a.moves[1 + 2 * m++] = i;
      if (!mover) a.remap[i] = use ? i : -1;
      if (a.refs_out != a.refs && !mover && !hole) a.refs_out[i] = n[u];
    }
    hat += s & 0xffff;
    mat += s >> 16;
  }
  if (gtid == 0) {
    *a.live = live;
    a.moves[0] = mtotal;
  }
  cluster_sync_all();
  for (int k = gtid; k < mtotal; k += gthreads) {
    const int from = __ldcg(a.moves + 1 + 2 * k), to = __ldcg(a.moves + 2 + 2 * k);
    a.remap[from] = to;
    a.refs_out[to] = a.refs[from];  // in place: `from` >= live > `to`, and each is touched once
    a.refs_out[from] = 0;
  }
}

// The moves' bytes and the tables: CTAs stride over (move, buffer) and over the table's cells.  Beside K and V up to two
// smaller buffers of whole words move (page bounds; an 8-bit cache's scales).
template <typename Chunk>
__global__ void __launch_bounds__(256) move_pages_kernel(unsigned char* kc, unsigned char* vc, unsigned char* side0,
                                                         unsigned char* side1, long long page_bytes, long long side_bytes,
                                                         const int32_t* __restrict__ moves,
                                                         const int32_t* __restrict__ remap, int num_blocks,
                                                         const int32_t* table, int32_t* table_out, long long cells,
                                                         int32_t* status) {
  pdl_wait();
  const int tid = threadIdx.x;
  for (long long i = blockIdx.x * 256LL + tid; i < cells; i += gridDim.x * 256LL) {
    const int p = table[i];
    int q = -1;
    if (p != -1) {
      if (p >= 0 && p < num_blocks) q = remap[p];
      if (q < 0) report(status, TS_ERR_DEVICE_CHECK);
    }
    table_out[i] = q;
  }
  const int n = moves[0], bufs = 2 + (side0 != nullptr) + (side1 != nullptr);
  for (long long it = blockIdx.x; it < static_cast<long long>(n) * bufs; it += gridDim.x) {
    const int k = static_cast<int>(it / bufs), which = static_cast<int>(it - static_cast<long long>(k) * bufs);
    const long long from = moves[1 + 2 * k], to = moves[2 + 2 * k];
    if (which >= 2) {
      unsigned char* side = which == 2 ? side0 : side1;
      const uint32_t* s = reinterpret_cast<const uint32_t*>(side + from * side_bytes);
      uint32_t* d = reinterpret_cast<uint32_t*>(side + to * side_bytes);
      for (long long i = tid; i < side_bytes / 4; i += 256) d[i] = s[i];
      continue;
    }
    unsigned char* base = which == 0 ? kc : vc;
    const Chunk* s = reinterpret_cast<const Chunk*>(base + from * page_bytes);
    Chunk* d = reinterpret_cast<Chunk*>(base + to * page_bytes);
    const int chunks = static_cast<int>(page_bytes / static_cast<long long>(sizeof(Chunk)));
    for (int i0 = tid; i0 < chunks; i0 += 256 * 8) {
      Chunk v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + 256 * u < chunks) v[u] = s[i0 + 256 * u];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + 256 * u < chunks) d[i0 + 256 * u] = v[u];
    }
  }
}

bool wide_rows(const void* k, const void* v, int row_bytes) {
  return row_bytes % 16 == 0 && ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) == 0;
}

long long most_requests(int num_blocks, int block_size, int B, int n) {
  const long long per_row = (static_cast<long long>(n) + block_size - 2) / block_size + 1;
  return std::min<long long>(num_blocks, per_row * B);
}

}  // namespace

size_t kv_reserve_workspace_bytes(int num_blocks, int block_size, int B, int n) {
  return 4 * (static_cast<size_t>(2) * B + static_cast<size_t>(most_requests(num_blocks, block_size, B, n)));
}

int kv_reserve_launch(const ReserveCall& c, cudaStream_t stream) {
  ReserveArgs a;
  a.table = c.block_table;
  a.prefix_len = c.prefix_len;
  a.refs = c.refs;
  a.freed = c.freed;
  a.table_out = c.block_table_out;
  a.refs_out = c.refs_out;
  a.granted = c.granted;
  a.copy = static_cast<int32_t*>(c.workspace);
  a.free_list = a.copy + 2 * static_cast<size_t>(c.B);
  a.status = c.dev_status;
  a.n = c.n;
  a.num_blocks = c.num_blocks;
  a.bs = c.block_size;
  a.max_blocks = c.max_blocks;
  a.B = c.B;
  a.num_freed = c.num_freed;
  cudaError_t e = launch_pdl(reserve_kernel, dim3(kPoolCtas), dim3(kPoolThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  const int row_bytes = c.d * c.elem_bytes;
  const Scales scales{c.k_scale, c.v_scale, c.k_scale != nullptr ? c.block_size / c.scale_block : 0};
  unsigned char *k = static_cast<unsigned char*>(c.k_cache), *v = static_cast<unsigned char*>(c.v_cache);
  const dim3 grid(c.Hkv, c.B);
  e = wide_rows(k, v, row_bytes)
          ? launch_pdl(copy_tails_kernel<uint4>, grid, dim3(256), 0, stream, k, v, c.Hkv, c.block_size, row_bytes, scales,
                       a.copy, c.prefix_len)
          : launch_pdl(copy_tails_kernel<uint32_t>, grid, dim3(256), 0, stream, k, v, c.Hkv, c.block_size, row_bytes, scales,
                       a.copy, c.prefix_len);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  return TS_OK;
}

int kv_fork_launch(const int32_t* block_table, int max_blocks, const int32_t* prefix_len, const int32_t* refs, int num_blocks,
                   int block_size, int B, const int32_t* src, int B_out, int32_t* block_table_out, int32_t* prefix_len_out,
                   int32_t* refs_out, int32_t* dev_status, cudaStream_t stream, int num_sms) {
  const ForkArgs a{block_table, prefix_len, refs, src, block_table_out, prefix_len_out, refs_out, dev_status,
                   max_blocks, num_blocks, block_size, B, B_out};
  // Up to some ten thousand words, one cluster does both steps with its own barrier between them: 6.3 us on the
  // device either way for one sequence becoming eight of 128 pages, and a launch less for the host (16.5 us a
  // call from Python against 19.4); larger states are spread over the GPU (512 rows of 512 pages: 8.3 us).
  const long long words = (static_cast<long long>(B) + B_out) * max_blocks + num_blocks;
  if (words <= 32768) {
    const cudaError_t e = launch_pdl(fork_small_kernel, dim3(kPoolCtas), dim3(kForkThreads), 0, stream, a);
    count_launches(1);
    return e == cudaSuccess ? TS_OK : TS_ERR_CUDA;
  }
  const int copy_ctas = refs_out != refs ? (num_blocks + 1023) / 1024 : 1;
  const int g1 = std::min(std::max(B_out, copy_ctas), 8 * num_sms);
  cudaError_t e = launch_pdl(fork_rows_kernel, dim3(g1), dim3(kForkThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  e = launch_pdl(fork_refs_kernel, dim3(std::min(B, 8 * num_sms)), dim3(kForkThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  return TS_OK;
}

size_t kv_compact_workspace_bytes(int num_blocks) { return 4 * (static_cast<size_t>(num_blocks) + 2); }

int kv_compact_launch(const CompactCall& c, cudaStream_t stream, int num_sms) {
  CompactArgs a{c.refs, c.refs_out, c.remap, c.live, static_cast<int32_t*>(c.workspace), c.num_blocks};
  cudaError_t e = launch_pdl(compact_kernel, dim3(kPoolCtas), dim3(kPoolThreads), 0, stream, a);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  unsigned char *k = static_cast<unsigned char*>(c.k_cache), *v = static_cast<unsigned char*>(c.v_cache);
  unsigned char *side0 = static_cast<unsigned char*>(c.side[0]), *side1 = static_cast<unsigned char*>(c.side[1]);
  const long long page_bytes = static_cast<long long>(c.Hkv) * c.block_size * c.row_bytes;
  const long long cells = static_cast<long long>(c.B) * c.max_blocks;
  const int bufs = 2 + (side0 != nullptr) + (side1 != nullptr);
  // A CTA per buffer of a move up to 64 per SM (6100 pages of 64 KB: 148 us against 160 with eight per SM), at most
  // what this pool can have.
  const long long most = std::max((cells + 255) / 256, (static_cast<long long>(c.num_blocks) / 2 + 1) * bufs);
  const dim3 grid(static_cast<unsigned>(std::min<long long>(64LL * num_sms, most)));
  e = wide_rows(k, v, c.row_bytes)
          ? launch_pdl(move_pages_kernel<uint4>, grid, dim3(256), 0, stream, k, v, side0, side1, page_bytes, c.side_bytes,
                       a.moves, c.remap, c.num_blocks, c.block_table, c.block_table_out, cells, c.dev_status)
          : launch_pdl(move_pages_kernel<uint32_t>, grid, dim3(256), 0, stream, k, v, side0, side1, page_bytes, c.side_bytes,
                       a.moves, c.remap, c.num_blocks, c.block_table, c.block_table_out, cells, c.dev_status);
  if (e != cudaSuccess) return TS_ERR_CUDA;
  count_launches(1);
  return TS_OK;
}

}  // namespace ts
