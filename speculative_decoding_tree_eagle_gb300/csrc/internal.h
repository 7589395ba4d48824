// Internal launch entry points behind the C ABI (host side).  Arguments are already
// validated by the C-ABI layer when these are called.
#pragma once

#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "treespec.h"

namespace ts {

int device_sm_count();

// Runs `set` (a kernel's attribute, which CUDA keeps per device) the first time the current device is seen;
// `done` holds a bit per device.  Several threads may run it at once, which does no harm.
template <typename F>
inline cudaError_t once_per_device(std::atomic<uint64_t>& done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if ((done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

size_t tree_build_workspace_bytes(int B, int V, int k, int depth, int num_sms);
int tree_build_launch(const float* draft_logp, const int32_t* root_tokens, int B, int V, int k,
                      int depth, int m, int32_t* tokens, int32_t* parents, int32_t* depth_out,
                      uint64_t* mask, double* values, int32_t* node_row, void* workspace, int32_t* dev_status,
                      cudaStream_t stream, int num_sms);

size_t tree_accept_workspace_bytes(ts_dtype dt, int B, int m, int V, int num_sms);
int tree_accept_launch(const void* logits, ts_dtype dt, const int32_t* tokens,
                       const int32_t* parents, int B, int m, int V, int32_t* argmax,
                       int32_t* accept_len, int32_t* accept_path, int32_t* bonus, void* workspace,
                       int32_t* dev_status, cudaStream_t stream, int num_sms);

struct AttnArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  ts_dtype dt;
  int num_blocks, block_size;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* prefix_len;
  int max_prefix;
  const uint64_t* mask;
  int B, m, Hq, Hkv, d;
  float scale;
  void* out;
  float* lse;
  void* workspace;
  int32_t* dev_status;
  cudaStream_t stream;
};

// Whether the tensor-core path handles this shape (bf16, d == 128, block size 16..128).
bool attention_uses_tc(ts_dtype dt, int d, int block_size);
size_t attention_tc_workspace_bytes(int B, int m, int Hq, int Hkv, int max_prefix, int num_sms);
int attention_tc_launch(const AttnArgs& a, int num_sms);
// {row groups of 128 rows, chunks, tiles per chunk, split mode, multicast width} of the
// tensor-core launch.
void attention_tc_plan(int B, int m, int Hq, int Hkv, int max_prefix, int num_sms, int* out5);
int attention_simt_launch(const AttnArgs& a);

// accept_kernel on precomputed per-row partials (value, index) [B*m, S].
int accept_from_partials_launch(const float* part_v, const int* part_i, int S, const int32_t* tokens,
                                const int32_t* parents, int B, int m, int32_t* argmax, int32_t* accept_len,
                                int32_t* accept_path, int32_t* bonus, int32_t* dev_status, cudaStream_t stream);

// LM-head GEMM with the per-row argmax in its epilogue (lm_head.cu).
size_t lm_head_partials(int M, int N, int num_sms);
size_t lm_head_workspace_bytes(int M, int N, int num_sms);
int lm_head_partials_launch(const void* hidden, const void* weight, int M, int N, int K, float* part_v,
                            int* part_i, int* S_out, int32_t* dev_status, cudaStream_t stream, int num_sms);
int lm_head_argmax_launch(const void* hidden, const void* weight, int M, int N, int K, int32_t* argmax,
                          float* max_logit, void* workspace, int32_t* dev_status, cudaStream_t stream,
                          int num_sms);

int tree_build_from_topk_launch(const int32_t* row_tok, const float* row_logp, const int32_t* root_tokens, int B,
                                int k, int depth, int m, int32_t* tokens, int32_t* parents, int32_t* depth_out,
                                uint64_t* mask, double* values, int32_t* node_row, int32_t* dev_status,
                                cudaStream_t stream);

// Stochastic verification by multi-round rejection sampling (tree_sample.cu).
size_t tree_accept_sample_workspace_bytes(int B, int V, int q_mode);
int tree_accept_sample_launch(const void* logits, ts_dtype dt, const int32_t* tokens, const int32_t* parents,
                              const float* uniforms, const float* draft_logp, const int32_t* node_row, int R,
                              int B, int m, int V, float temperature, int q_mode, int32_t* accept_len,
                              int32_t* accept_path, int32_t* bonus, void* workspace, int32_t* dev_status,
                              cudaStream_t stream);

// Cost-aware pruning before verification (tree_prune.cu).
size_t tree_prune_workspace_bytes(int B, int m);
int tree_prune_launch(const int32_t* tokens, const int32_t* parents, const int32_t* depth, const double* values,
                      const int32_t* node_row, int B, int m, double t_draft, double t_fixed, double t_node,
                      int32_t* n_out, int32_t* tokens_out, int32_t* parents_out, int32_t* depth_out, uint64_t* mask_out,
                      double* values_out, int32_t* node_row_out, int32_t* kept_out, float* expected_out,
                      void* workspace, int32_t* dev_status, cudaStream_t stream);

// Bounded-wait self-test (selftest.cu).
int selftest_bounded_wait_launch(int mode, int32_t* result, int32_t* dev_status, cudaStream_t stream);

int efficient_head_candidates(int V, int tile_tokens, int k_tile);
size_t efficient_head_workspace_bytes(int M, int V, int rank, int tile_tokens, int k_tile);
int efficient_head_launch(const void* hidden, const void* lr_b, const void* lr_a, const void* weight, int M, int V,
                          int d, int rank, int tile_tokens, int k_tile, int k, int32_t* top_tok, float* top_logp,
                          int32_t* cand_out, void* workspace, int32_t* dev_status, cudaStream_t stream,
                          int num_sms);

int kv_commit_launch(void* k_cache, void* v_cache, ts_dtype dt, int num_blocks, int block_size,
                     int Hkv, int d, int32_t* block_table, int max_blocks, int32_t* prefix_len,
                     const int32_t* accept_path, const int32_t* accept_len, int B, int m,
                     int32_t* freed_blocks, int32_t* freed_count, int32_t* dev_status,
                     cudaStream_t stream);

// Page bounds, the choice of pages and attention over it (page_bounds.cu, page_select.cu,
// tree_attention_tc.cu / tree_attention_sparse.cu).
int kv_page_bounds_launch(const void* k_cache, ts_dtype dt, int num_blocks, int block_size, int Hkv, int d,
                          const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                          const int32_t* start_len, int B, void* bounds, int32_t* dev_status, cudaStream_t stream,
                          int num_sms);

struct SelectCall {
  const void* q;
  ts_dtype dt;
  const void* bounds;
  int num_blocks, block_size;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* prefix_len;
  int max_prefix, B, m, Hq, Hkv, d, n_pages, first, recent;
  int32_t* pages;
  int32_t* count;
  uint64_t* node_mask;
  void* workspace;
  int32_t* dev_status;
};
size_t page_select_workspace_bytes(int B, int m, int Hq, int Hkv, int d, int C);
int page_select_launch(const SelectCall& c, cudaStream_t stream, int num_sms);

struct SparseCall {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  ts_dtype dt;
  int num_blocks, block_size;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* prefix_len;
  const uint64_t* mask;
  const int32_t* pages;
  const int32_t* count;
  const uint64_t* node_mask;
  int C, B, m, Hq, Hkv, d;
  float scale;
  void* out;
  float* lse;
  void* workspace;
  int32_t* dev_status;
};
int attention_sparse_simt_launch(const SparseCall& a, cudaStream_t stream, int num_sms);
size_t attention_sparse_tc_workspace_bytes(int B, int m, int Hq, int Hkv, int C, int block_size, int num_sms);
int attention_sparse_tc_launch(const SparseCall& a, cudaStream_t stream, int num_sms);

// The page pool (page_pool.cu).
struct ReserveCall {
  void* k_cache;
  void* v_cache;
  ts_dtype dt;
  int num_blocks, block_size, Hkv, d;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* prefix_len;
  const int32_t* refs;
  int B, n;
  const int32_t* freed;
  int num_freed;
  int32_t* block_table_out;
  int32_t* refs_out;
  int32_t* granted;
  void* workspace;
  int32_t* dev_status;
};
size_t kv_reserve_workspace_bytes(int num_blocks, int block_size, int B, int n);
int kv_reserve_launch(const ReserveCall& c, cudaStream_t stream);
int kv_fork_launch(const int32_t* block_table, int max_blocks, const int32_t* prefix_len, const int32_t* refs, int num_blocks,
                   int block_size, int B, const int32_t* src, int B_out, int32_t* block_table_out, int32_t* prefix_len_out,
                   int32_t* refs_out, int32_t* dev_status, cudaStream_t stream, int num_sms);
size_t kv_compact_workspace_bytes(int num_blocks);
int kv_compact_launch(void* k_cache, void* v_cache, ts_dtype dt, void* bounds, int num_blocks, int block_size, int Hkv, int d,
                      const int32_t* block_table, int max_blocks, const int32_t* refs, int B, int32_t* block_table_out,
                      int32_t* refs_out, int32_t* remap, int32_t* live, void* workspace, int32_t* dev_status,
                      cudaStream_t stream, int num_sms);

}  // namespace ts
