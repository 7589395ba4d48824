// C ABI of libtreespec.so (declared in include/treespec.h): host-side argument validation,
// workspace sizing and dispatch to the kernels.  Nothing here allocates device memory.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "common.cuh"
#include "internal.h"

namespace ts {

static std::atomic<uint64_t> g_launches{0};

void count_launches(int n) { g_launches.fetch_add(static_cast<uint64_t>(n), std::memory_order_relaxed); }

int device_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int check_build(int B, int V, int k, int depth, int m) {
  if (B <= 0 || V <= 0 || k <= 0 || depth <= 0 || m <= 0) return TS_ERR_INVALID;
  if (k > TS_MAX_TOPK || depth > TS_MAX_DEPTH || m > TS_MAX_NODES) return TS_ERR_UNSUPPORTED;
  if (k > V) return TS_ERR_INVALID;
  const long long ncand = k + static_cast<long long>(depth - 1) * k * k;
  if (m - 1 > ncand) return TS_ERR_INVALID;
  const long long R = 1 + static_cast<long long>(depth - 1) * k;
  if (static_cast<long long>(B) * R * V > (1LL << 40)) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

static int check_attention(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int max_prefix) {
  if (B <= 0 || m <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || max_prefix < 0) return TS_ERR_INVALID;
  if (dt != TS_F32 && dt != TS_BF16) return TS_ERR_INVALID;
  if (Hq % Hkv != 0) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES || d > 256 || static_cast<long long>(B) * Hkv > 65535)
    return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

static int check_accept(ts_dtype dt, int B, int m, int V) {
  if (B <= 0 || m <= 0 || V <= 0) return TS_ERR_INVALID;
  if (dt != TS_F32 && dt != TS_BF16) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

}  // namespace ts

// A tensor's memory, as the checks for overlap see it (size 0 where a tensor is left out).
struct Memory {
  uintptr_t at;
  size_t size;
  Memory(const void* p, size_t elems, size_t elem_size) : at(reinterpret_cast<uintptr_t>(p)), size(p ? elems * elem_size : 0) {}
};
static bool overlap(const Memory& a, const Memory& b) {
  return a.size > 0 && b.size > 0 && a.at < b.at + b.size && b.at < a.at + a.size;
}
// Whether every output lies apart from the inputs and from the other outputs; an output that may be its input's buffer
// and is leaves that input out.
static bool outputs_apart(std::initializer_list<Memory> outs, std::initializer_list<Memory> ins) {
  for (const Memory* o = outs.begin(); o != outs.end(); ++o) {
    for (const Memory& i : ins)
      if (overlap(*o, i)) return false;
    for (const Memory* other = o + 1; other != outs.end(); ++other)
      if (overlap(*o, *other)) return false;
  }
  return true;
}
static size_t times(int a, int b, int c = 1, int d = 1) {
  return static_cast<size_t>(a) * static_cast<size_t>(b) * static_cast<size_t>(c) * static_cast<size_t>(d);
}

static bool aligned4_ptr(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool aligned16_ptr(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

extern "C" {

const char* ts_status_string(int status) {
  switch (status) {
    case TS_OK: return "TS_OK";
    case TS_ERR_INVALID: return "TS_ERR_INVALID: invalid argument";
    case TS_ERR_UNSUPPORTED: return "TS_ERR_UNSUPPORTED: size outside the supported range";
    case TS_ERR_WORKSPACE: return "TS_ERR_WORKSPACE: workspace too small";
    case TS_ERR_CUDA: return "TS_ERR_CUDA: CUDA launch or driver call failed";
    case TS_ERR_TIMEOUT: return "TS_ERR_TIMEOUT: a bounded device wait timed out";
    case TS_ERR_DEVICE_CHECK: return "TS_ERR_DEVICE_CHECK: bad input data found on the device";
    case TS_ERR_NO_PAGES: return "TS_ERR_NO_PAGES: the page pool has too few free pages";
    default: return "unknown ts_status";
  }
}

int ts_version(void) { return 1; }

uint64_t ts_launch_count(void) { return ts::g_launches.load(std::memory_order_relaxed); }

size_t ts_tree_build_workspace(int B, int V, int k, int depth, int m) {
  if (ts::check_build(B, V, k, depth, m) != TS_OK) return 0;
  return ts::tree_build_workspace_bytes(B, V, k, depth, ts::device_sm_count());
}

int ts_tree_build(const float* draft_logp, const int32_t* root_tokens, int B, int V, int k,
                  int depth, int m, int32_t* tokens, int32_t* parents, int32_t* depth_out,
                  uint64_t* mask, double* values, int32_t* node_row, void* workspace, size_t ws_bytes,
                  int32_t* dev_status, void* stream) {
  const int rc = ts::check_build(B, V, k, depth, m);
  if (rc != TS_OK) return rc;
  if (!draft_logp || !root_tokens || !tokens || !parents || !depth_out || !mask || !workspace)
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  if (ws_bytes < ts::tree_build_workspace_bytes(B, V, k, depth, sms)) return TS_ERR_WORKSPACE;
  return ts::tree_build_launch(draft_logp, root_tokens, B, V, k, depth, m, tokens, parents,
                               depth_out, mask, values, node_row, workspace, dev_status,
                               static_cast<cudaStream_t>(stream), sms);
}

size_t ts_tree_attention_workspace(ts_dtype dt, int B, int m, int Hq, int Hkv, int d,
                                   int max_prefix) {
  if (ts::check_attention(dt, B, m, Hq, Hkv, d, max_prefix) != TS_OK) return 0;
  if (ts::attention_uses_tc(dt, d, 16))
    return ts::attention_tc_workspace_bytes(B, m, Hq, Hkv, max_prefix, ts::device_sm_count());
  return 256;
}

// num_sms <= 0: the current device's SM count, looked up only for the tensor-core path
static int attention_plan(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int max_prefix,
                          int block_size, int num_sms, int* plan_out) {
  const int rc = ts::check_attention(dt, B, m, Hq, Hkv, d, max_prefix);
  if (rc != TS_OK) return rc;
  if (!plan_out || block_size <= 0) return TS_ERR_INVALID;
  if (!ts::attention_uses_tc(dt, d, block_size)) {
    plan_out[0] = 0;
    plan_out[1] = 0;
    plan_out[2] = 1;
    plan_out[3] = 0;
    plan_out[4] = 0;
    plan_out[5] = 1;
    return TS_OK;
  }
  plan_out[0] = 1;
  ts::attention_tc_plan(B, m, Hq, Hkv, max_prefix, num_sms > 0 ? num_sms : ts::device_sm_count(), plan_out + 1);
  return TS_OK;
}

int ts_tree_attention_plan(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int max_prefix,
                           int block_size, int* plan_out) {
  return attention_plan(dt, B, m, Hq, Hkv, d, max_prefix, block_size, 0, plan_out);
}

int ts_tree_attention_plan_for_sms(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int max_prefix,
                                   int block_size, int num_sms, int* plan_out) {
  if (num_sms < 1) return TS_ERR_INVALID;
  return attention_plan(dt, B, m, Hq, Hkv, d, max_prefix, block_size, num_sms, plan_out);
}

int ts_tree_attention(const void* q, const void* k_cache, const void* v_cache, ts_dtype dt,
                      int num_blocks, int block_size, const int32_t* block_table,
                      int max_blocks, const int32_t* prefix_len, int max_prefix,
                      const uint64_t* mask, int B, int m, int Hq, int Hkv, int d,
                      float scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                      int32_t* dev_status, void* stream) {
  int rc = ts::check_attention(dt, B, m, Hq, Hkv, d, max_prefix);
  if (rc != TS_OK) return rc;
  if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !mask || !out)
    return TS_ERR_INVALID;
  if (num_blocks <= 0 || block_size <= 0 || max_blocks <= 0 || !std::isfinite(scale))
    return TS_ERR_INVALID;
  if (static_cast<long long>(max_blocks) * block_size < static_cast<long long>(max_prefix) + m)
    return TS_ERR_INVALID;
  ts::AttnArgs a{q, k_cache, v_cache, dt, num_blocks, block_size, block_table, max_blocks,
                 prefix_len, max_prefix, mask, B, m, Hq, Hkv, d, scale, out, lse, workspace,
                 dev_status, static_cast<cudaStream_t>(stream)};
  if (ts::attention_uses_tc(dt, d, block_size)) {
    if (!ts::aligned16(q) || !ts::aligned16(k_cache) || !ts::aligned16(v_cache) || !ts::aligned16(out))
      return TS_ERR_INVALID;
    const int sms = ts::device_sm_count();
    if (sms <= 0) return TS_ERR_CUDA;
    const size_t need = ts::attention_tc_workspace_bytes(B, m, Hq, Hkv, max_prefix, sms);
    if (need > 256 && (!workspace || ws_bytes < need)) return TS_ERR_WORKSPACE;
    if (!ts::aligned16(workspace) && need > 256) return TS_ERR_INVALID;
    return ts::attention_tc_launch(a, sms);
  }
  return ts::attention_simt_launch(a);
}

size_t ts_tree_accept_workspace(ts_dtype dt, int B, int m, int V) {
  if (ts::check_accept(dt, B, m, V) != TS_OK) return 0;
  return ts::tree_accept_workspace_bytes(dt, B, m, V, ts::device_sm_count());
}

int ts_tree_accept(const void* logits, ts_dtype dt, const int32_t* tokens,
                   const int32_t* parents, int B, int m, int V, int32_t* argmax,
                   int32_t* accept_len, int32_t* accept_path, int32_t* bonus, void* workspace,
                   size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int rc = ts::check_accept(dt, B, m, V);
  if (rc != TS_OK) return rc;
  if (!logits || !tokens || !parents || !argmax || !accept_len || !accept_path || !bonus ||
      !workspace)
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  if (ws_bytes < ts::tree_accept_workspace_bytes(dt, B, m, V, sms)) return TS_ERR_WORKSPACE;
  return ts::tree_accept_launch(logits, dt, tokens, parents, B, m, V, argmax, accept_len,
                                accept_path, bonus, workspace, dev_status,
                                static_cast<cudaStream_t>(stream), sms);
}

static int check_lm_head(const void* hidden, const void* weight, long long M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 8 != 0) return TS_ERR_INVALID;
  if (!hidden || !weight || !aligned16_ptr(hidden) || !aligned16_ptr(weight)) return TS_ERR_INVALID;
  if (M > (1LL << 24)) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

size_t ts_lm_head_argmax_workspace(int M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 8 != 0) return 0;
  return ts::lm_head_workspace_bytes(M, N, ts::device_sm_count());
}

int ts_lm_head_argmax(const void* hidden, const void* weight, int M, int N, int K, int32_t* argmax,
                      float* max_logit, void* workspace, size_t ws_bytes, int32_t* dev_status,
                      void* stream) {
  const int rc = check_lm_head(hidden, weight, M, N, K);
  if (rc != TS_OK) return rc;
  if (!argmax || !workspace) return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  if (ws_bytes < ts::lm_head_workspace_bytes(M, N, sms)) return TS_ERR_WORKSPACE;
  return ts::lm_head_argmax_launch(hidden, weight, M, N, K, argmax, max_logit, workspace, dev_status,
                                   static_cast<cudaStream_t>(stream), sms);
}

size_t ts_tree_accept_hidden_workspace(int B, int m, int V, int K) {
  if (B <= 0 || m <= 0 || m > TS_MAX_NODES) return 0;
  return ts_lm_head_argmax_workspace(B * m, V, K);
}

int ts_tree_accept_hidden(const void* hidden, const void* weight, const int32_t* tokens,
                          const int32_t* parents, int B, int m, int V, int K, int32_t* argmax,
                          int32_t* accept_len, int32_t* accept_path, int32_t* bonus, void* workspace,
                          size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (B <= 0 || m <= 0) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES) return TS_ERR_UNSUPPORTED;
  const long long M = static_cast<long long>(B) * m;
  const int rc = check_lm_head(hidden, weight, M, V, K);
  if (rc != TS_OK) return rc;
  if (!tokens || !parents || !argmax || !accept_len || !accept_path || !bonus || !workspace)
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  const int Mi = static_cast<int>(M);
  if (ws_bytes < ts::lm_head_workspace_bytes(Mi, V, sms)) return TS_ERR_WORKSPACE;
  const int G = static_cast<int>(ts::lm_head_partials(Mi, V, sms));
  float* part_v = static_cast<float*>(workspace);
  int* part_i = reinterpret_cast<int*>(part_v + M * G);
  int S = 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int r1 = ts::lm_head_partials_launch(hidden, weight, Mi, V, K, part_v, part_i, &S, dev_status, st, sms);
  if (r1 != TS_OK) return r1;
  return ts::accept_from_partials_launch(part_v, part_i, S, tokens, parents, B, m, argmax, accept_len,
                                         accept_path, bonus, dev_status, st);
}

int ts_efficient_head_candidates(int V, int tile_tokens, int k_tile) {
  if (V <= 0 || tile_tokens <= 0 || tile_tokens % 256 != 0 || k_tile < 1 || k_tile > 8) return 0;
  return ts::efficient_head_candidates(V, tile_tokens, k_tile);
}

static int check_efficient_head(const void* hidden, const void* lr_b, const void* lr_a, const void* weight, int M,
                                int V, int d, int rank, int tile_tokens, int k_tile, int k) {
  if (M <= 0 || V <= 0 || d <= 0 || rank <= 0 || d % 8 != 0 || rank % 8 != 0) return TS_ERR_INVALID;
  if (tile_tokens <= 0 || tile_tokens % 256 != 0 || k_tile < 1 || k_tile > tile_tokens) return TS_ERR_INVALID;
  if (k_tile > 8 || k < 1 || k > TS_MAX_TOPK) return TS_ERR_UNSUPPORTED;
  const long long C = static_cast<long long>((V + tile_tokens - 1) / tile_tokens) * k_tile;
  if (k > C) return TS_ERR_INVALID;
  if (C * 8 > 200 * 1024 || M > 65535) return TS_ERR_UNSUPPORTED;
  if (!hidden || !lr_b || !lr_a || !weight) return TS_ERR_INVALID;
  if (!aligned16_ptr(hidden) || !aligned16_ptr(lr_b) || !aligned16_ptr(lr_a) || !aligned16_ptr(weight))
    return TS_ERR_INVALID;
  return TS_OK;
}

size_t ts_efficient_head_workspace(int M, int V, int d, int rank, int tile_tokens, int k_tile) {
  const void* p = reinterpret_cast<const void*>(static_cast<uintptr_t>(256));
  if (check_efficient_head(p, p, p, p, M, V, d, rank, tile_tokens, k_tile, 1) != TS_OK) return 0;
  return ts::efficient_head_workspace_bytes(M, V, rank, tile_tokens, k_tile);
}

int ts_efficient_head(const void* hidden, const void* lr_b, const void* lr_a, const void* weight, int M,
                      int V, int d, int rank, int tile_tokens, int k_tile, int k, int32_t* top_tok,
                      float* top_logp, int32_t* candidates, void* workspace, size_t ws_bytes,
                      int32_t* dev_status, void* stream) {
  const int rc = check_efficient_head(hidden, lr_b, lr_a, weight, M, V, d, rank, tile_tokens, k_tile, k);
  if (rc != TS_OK) return rc;
  if (!top_tok || !top_logp || !workspace) return TS_ERR_INVALID;
  if (ws_bytes < ts::efficient_head_workspace_bytes(M, V, rank, tile_tokens, k_tile)) return TS_ERR_WORKSPACE;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  return ts::efficient_head_launch(hidden, lr_b, lr_a, weight, M, V, d, rank, tile_tokens, k_tile, k, top_tok,
                                   top_logp, candidates, workspace, dev_status, static_cast<cudaStream_t>(stream),
                                   sms);
}

int ts_tree_build_from_topk(const int32_t* row_tok, const float* row_logp, const int32_t* root_tokens,
                            int B, int k, int depth, int m, int32_t* tokens, int32_t* parents,
                            int32_t* depth_out, uint64_t* mask, double* values, int32_t* node_row,
                            int32_t* dev_status, void* stream) {
  if (B <= 0 || k <= 0 || depth <= 0 || m <= 0) return TS_ERR_INVALID;
  if (k > TS_MAX_TOPK || depth > TS_MAX_DEPTH || m > TS_MAX_NODES) return TS_ERR_UNSUPPORTED;
  const long long ncand = k + static_cast<long long>(depth - 1) * k * k;
  if (m - 1 > ncand) return TS_ERR_INVALID;
  if (!row_tok || !row_logp || !root_tokens || !tokens || !parents || !depth_out || !mask) return TS_ERR_INVALID;
  return ts::tree_build_from_topk_launch(row_tok, row_logp, root_tokens, B, k, depth, m, tokens, parents, depth_out,
                                         mask, values, node_row, dev_status, static_cast<cudaStream_t>(stream));
}

int ts_kv_commit(void* k_cache, void* v_cache, ts_dtype dt, int num_blocks, int block_size,
                 int Hkv, int d, int32_t* block_table, int max_blocks, int32_t* prefix_len,
                 const int32_t* accept_path, const int32_t* accept_len, int B, int m,
                 int32_t* freed_blocks, int32_t* freed_count, int32_t* dev_status, void* stream) {
  if (B <= 0 || m <= 0 || num_blocks <= 0 || block_size <= 0 || Hkv <= 0 || d <= 0 || max_blocks <= 0)
    return TS_ERR_INVALID;
  if (dt != TS_F32 && dt != TS_BF16) return TS_ERR_INVALID;
  if ((d * (dt == TS_BF16 ? 2 : 4)) % 4 != 0) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES || B > 65535) return TS_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !block_table || !prefix_len || !accept_path || !accept_len ||
      !freed_blocks || !freed_count)
    return TS_ERR_INVALID;
  return ts::kv_commit_launch(k_cache, v_cache, dt, num_blocks, block_size, Hkv, d, block_table,
                              max_blocks, prefix_len, accept_path, accept_len, B, m, freed_blocks,
                              freed_count, dev_status, static_cast<cudaStream_t>(stream));
}

size_t ts_tree_accept_sample_workspace(int B, int V, int q_mode) {
  if (B <= 0 || V <= 0 || (q_mode != TS_Q_POINT && q_mode != TS_Q_DRAFT)) return 0;
  return ts::tree_accept_sample_workspace_bytes(B, V, q_mode);
}

int ts_tree_accept_sample(const void* logits, ts_dtype dt, const int32_t* tokens, const int32_t* parents,
                          const float* uniforms, const float* draft_logp, const int32_t* node_row, int R,
                          int B, int m, int V, float temperature, int q_mode, int32_t* accept_len,
                          int32_t* accept_path, int32_t* bonus, void* workspace, size_t ws_bytes,
                          int32_t* dev_status, void* stream) {
  if (B <= 0 || m <= 0 || V <= 0) return TS_ERR_INVALID;
  if (dt != TS_F32 && dt != TS_BF16) return TS_ERR_INVALID;
  if (q_mode != TS_Q_POINT && q_mode != TS_Q_DRAFT) return TS_ERR_INVALID;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES || V > TS_SAMPLE_MAX_VOCAB || B > 65535) return TS_ERR_UNSUPPORTED;
  if (!logits || !tokens || !parents || !uniforms || !accept_len || !accept_path || !bonus) return TS_ERR_INVALID;
  if (q_mode == TS_Q_DRAFT && (!draft_logp || !node_row || R <= 0)) return TS_ERR_INVALID;
  const size_t need = ts::tree_accept_sample_workspace_bytes(B, V, q_mode);
  if (need > 0 && (!workspace || ws_bytes < need)) return workspace ? TS_ERR_WORKSPACE : TS_ERR_INVALID;
  return ts::tree_accept_sample_launch(logits, dt, tokens, parents, uniforms, draft_logp, node_row, R, B, m, V,
                                       temperature, q_mode, accept_len, accept_path, bonus, workspace, dev_status,
                                       static_cast<cudaStream_t>(stream));
}

size_t ts_tree_prune_workspace(int B, int m) {
  if (B <= 0 || m <= 0 || m > TS_MAX_NODES) return 0;
  return ts::tree_prune_workspace_bytes(B, m);
}

int ts_tree_prune(const int32_t* tokens, const int32_t* parents, const int32_t* depth, const double* values,
                  const int32_t* node_row, int B, int m, double t_draft, double t_fixed, double t_node,
                  int32_t* n_out, int32_t* tokens_out, int32_t* parents_out, int32_t* depth_out,
                  uint64_t* mask_out, double* values_out, int32_t* node_row_out, int32_t* kept_out,
                  float* expected_out, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (B <= 0 || m <= 0) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES || B > 65535) return TS_ERR_UNSUPPORTED;
  if (!(t_draft >= 0.0) || !(t_fixed >= 0.0) || !(t_node >= 0.0) || !std::isfinite(t_draft) ||
      !std::isfinite(t_fixed) || !std::isfinite(t_node) || !(t_draft + t_fixed + t_node > 0.0))
    return TS_ERR_INVALID;
  if (!tokens || !parents || !depth || !values || !n_out || !tokens_out || !parents_out || !depth_out || !mask_out ||
      !values_out || !kept_out || !expected_out || !workspace)
    return TS_ERR_INVALID;
  if (node_row_out && !node_row) return TS_ERR_INVALID;
  if (ws_bytes < ts::tree_prune_workspace_bytes(B, m)) return TS_ERR_WORKSPACE;
  return ts::tree_prune_launch(tokens, parents, depth, values, node_row, B, m, t_draft, t_fixed, t_node, n_out,
                               tokens_out, parents_out, depth_out, mask_out, values_out, node_row_out, kept_out,
                               expected_out, workspace, dev_status, static_cast<cudaStream_t>(stream));
}

// What the calls on a paged cache share.
static int check_cache(ts_dtype dt, int num_blocks, int block_size, int Hkv, int d, int max_blocks, int B) {
  if (dt != TS_F32 && dt != TS_BF16) return TS_ERR_INVALID;
  if (num_blocks <= 0 || block_size <= 0 || Hkv <= 0 || d <= 0 || max_blocks <= 0 || B <= 0) return TS_ERR_INVALID;
  if (B > 65535) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

int ts_kv_page_bounds(const void* k_cache, ts_dtype dt, int num_blocks, int block_size, int Hkv, int d,
                      const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                      const int32_t* start_len, int B, void* bounds, int32_t* dev_status, void* stream) {
  const int rc = check_cache(dt, num_blocks, block_size, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (d > 256) return TS_ERR_UNSUPPORTED;
  if (!k_cache || !block_table || !prefix_len || !bounds) return TS_ERR_INVALID;
  const size_t size = dt == TS_BF16 ? 2 : 4;
  if (!outputs_apart({{bounds, times(num_blocks, Hkv, 2, d), 2}},
                     {{k_cache, times(num_blocks, Hkv, block_size, d), size},
                      {block_table, times(B, max_blocks), 4},
                      {prefix_len, times(B, 1), 4},
                      {start_len, times(B, 1), 4}}))
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  return ts::kv_page_bounds_launch(k_cache, dt, num_blocks, block_size, Hkv, d, block_table, max_blocks, prefix_len,
                                   start_len, B, bounds, dev_status, static_cast<cudaStream_t>(stream), sms);
}

static int check_select(int B, int m, int Hq, int Hkv, int d, int max_prefix, int block_size) {
  if (B <= 0 || m <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || max_prefix < 0 || block_size <= 0 || Hq % Hkv != 0)
    return TS_ERR_INVALID;
  if (m > TS_MAX_NODES || d > 256 || Hq / Hkv > 128 || max_prefix / block_size > 65536 ||
      static_cast<long long>(B) * Hkv > 65535)
    return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

size_t ts_page_select_workspace(int B, int m, int Hq, int Hkv, int d, int max_prefix, int block_size) {
  if (check_select(B, m, Hq, Hkv, d, max_prefix, block_size) != TS_OK) return 0;
  const int C = max_prefix / block_size;
  return ts::page_select_workspace_bytes(B, m, Hq, Hkv, d, C > 0 ? C : 1);
}

int ts_page_select(const void* q, ts_dtype dt, const void* bounds, int num_blocks, int block_size,
                   const int32_t* block_table, int max_blocks, const int32_t* prefix_len, int max_prefix,
                   int B, int m, int Hq, int Hkv, int d, int n_pages, int first, int recent,
                   int32_t* pages, int32_t* count, uint64_t* node_mask,
                   void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  int rc = check_select(B, m, Hq, Hkv, d, max_prefix, block_size);
  if (rc != TS_OK) return rc;
  rc = check_cache(dt, num_blocks, block_size, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (n_pages < 1 || first < 0 || recent < 0 || static_cast<long long>(first) + recent > n_pages) return TS_ERR_INVALID;
  if (static_cast<long long>(max_blocks) * block_size < max_prefix / block_size * static_cast<long long>(block_size))
    return TS_ERR_INVALID;
  if (!q || !bounds || !block_table || !prefix_len || !pages || !count || !node_mask) return TS_ERR_INVALID;
  if (!aligned16_ptr(bounds)) return TS_ERR_INVALID;
  const size_t need = ts_page_select_workspace(B, m, Hq, Hkv, d, max_prefix, block_size);
  if (need > 256 && (!workspace || !aligned16_ptr(workspace))) return TS_ERR_INVALID;
  if (need > 256 && ws_bytes < need) return TS_ERR_WORKSPACE;
  const size_t places = times(B, Hkv, std::max(1, max_prefix / block_size)), size = dt == TS_BF16 ? 2 : 4;
  if (!outputs_apart({{pages, places, 4},
                      {count, times(B, Hkv), 4},
                      {node_mask, places * ((m + 63) / 64), 8},
                      {need > 256 ? workspace : nullptr, need, 1}},
                     {{q, times(B, m, Hq, d), size},
                      {bounds, times(num_blocks, Hkv, 2, d), 2},
                      {block_table, times(B, max_blocks), 4},
                      {prefix_len, times(B, 1), 4}}))
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  ts::SelectCall c{q, dt, bounds, num_blocks, block_size, block_table, max_blocks, prefix_len, max_prefix, B, m, Hq, Hkv, d,
                   n_pages, first, recent, pages, count, node_mask, workspace, dev_status};
  return ts::page_select_launch(c, static_cast<cudaStream_t>(stream), sms);
}

static int check_sparse(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int C, int block_size) {
  const int rc = ts::check_attention(dt, B, m, Hq, Hkv, d, 0);
  if (rc != TS_OK) return rc;
  if (C <= 0 || block_size <= 0) return TS_ERR_INVALID;
  // keys a node can have at most, as a 32-bit position
  if (static_cast<long long>(C) * block_size > (1LL << 30)) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

size_t ts_tree_attention_sparse_workspace(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int C, int block_size) {
  if (check_sparse(dt, B, m, Hq, Hkv, d, C, block_size) != TS_OK) return 0;
  if (ts::attention_uses_tc(dt, d, block_size))
    return ts::attention_sparse_tc_workspace_bytes(B, m, Hq, Hkv, C, block_size, ts::device_sm_count());
  return 256;
}

int ts_tree_attention_sparse(const void* q, const void* k_cache, const void* v_cache, ts_dtype dt,
                             int num_blocks, int block_size, const int32_t* block_table, int max_blocks,
                             const int32_t* prefix_len, const uint64_t* mask, const int32_t* pages,
                             const int32_t* count, const uint64_t* node_mask, int C,
                             int B, int m, int Hq, int Hkv, int d, float scale, void* out, float* lse,
                             void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  int rc = check_sparse(dt, B, m, Hq, Hkv, d, C, block_size);
  if (rc != TS_OK) return rc;
  rc = check_cache(dt, num_blocks, block_size, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !mask || !pages || !count || !node_mask || !out)
    return TS_ERR_INVALID;
  if (!std::isfinite(scale) || !(scale > 0.f)) return TS_ERR_INVALID;
  const size_t rows = times(B, m, Hq), size = dt == TS_BF16 ? 2 : 4, cache = times(num_blocks, Hkv, block_size, d);
  const size_t words = (m + 63) / 64, places = times(B, Hkv, C);
  auto apart = [&](size_t used) {  // with the bytes of the workspace that are used
    return outputs_apart({{out, rows * d, size}, {lse, rows, 4}, {workspace, used, 1}},
                         {{q, rows * d, size},  // (rows computed again read it after others have been written)
                          {k_cache, cache, size},
                          {v_cache, cache, size},
                          {block_table, times(B, max_blocks), 4},
                          {prefix_len, times(B, 1), 4},
                          {mask, times(B, m) * words, 8},
                          {pages, places, 4},
                          {count, times(B, Hkv), 4},
                          {node_mask, places * words, 8}});
  };
  if (!apart(0)) return TS_ERR_INVALID;
  ts::SparseCall a{q, k_cache, v_cache, dt, num_blocks, block_size, block_table, max_blocks, prefix_len, mask, pages, count,
                   node_mask, C, B, m, Hq, Hkv, d, scale, out, lse, workspace, dev_status};
  const int sms = ts::device_sm_count();
  if (!ts::attention_uses_tc(dt, d, block_size)) {
    if (Hq > 65535) return TS_ERR_UNSUPPORTED;
    if (sms <= 0) return TS_ERR_CUDA;
    return ts::attention_sparse_simt_launch(a, static_cast<cudaStream_t>(stream), sms);
  }
  if (!aligned16_ptr(q) || !aligned16_ptr(k_cache) || !aligned16_ptr(v_cache) || !aligned16_ptr(out)) return TS_ERR_INVALID;
  if (sms <= 0) return TS_ERR_CUDA;
  const size_t need = ts::attention_sparse_tc_workspace_bytes(B, m, Hq, Hkv, C, block_size, sms);
  if (need > 256 && (!workspace || ws_bytes < need)) return TS_ERR_WORKSPACE;
  if (need > 256 && (!aligned16_ptr(workspace) || !apart(need))) return TS_ERR_INVALID;
  return ts::attention_sparse_tc_launch(a, static_cast<cudaStream_t>(stream), sms);
}

// What the calls on 8-bit caches share.
static int check_fp8(int num_blocks, int block_size, int scale_block, int Hkv, int d, int max_blocks, int B) {
  const int rc = check_cache(TS_F32, num_blocks, block_size, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (scale_block <= 0 || block_size % scale_block != 0) return TS_ERR_INVALID;
  if (d > 256 || Hkv > 65535 / 2) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}
// The calls that quantise count a scale block's elements in 32 bits, by up to 256 at a time.
static bool block_counts(int scale_block, int d) { return static_cast<long long>(scale_block) * d <= INT32_MAX - 256; }
// The pool's 8-bit forms write pages of all four: they lie apart.
static bool fp8_scales(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int num_blocks, int block_size,
                       int scale_block, int Hkv, int d) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !aligned4_ptr(k_scale) || !aligned4_ptr(v_scale)) return false;
  const size_t cache = times(num_blocks, Hkv, block_size, d), scales = times(num_blocks, Hkv, block_size / scale_block);
  return outputs_apart({{k_cache, cache, 1}, {v_cache, cache, 1}, {k_scale, scales, 4}, {v_scale, scales, 4}}, {});
}
// Elements from a strided tensor's first to its last, and one.
static size_t extent(const int64_t* strides, int B, int n, int Hkv, int d) {
  return static_cast<size_t>((B - 1) * strides[0] + (n - 1) * strides[1] + (Hkv - 1) * strides[2] + d);
}

int ts_kv_write_fp8(const void* k, const void* v, ts_dtype dt, const int64_t* k_strides, const int64_t* v_strides, void* k_cache,
                    void* v_cache, float* k_scale, float* v_scale, int num_blocks, int block_size, int scale_block, int Hkv,
                    int d, const int32_t* block_table, int max_blocks, const int32_t* start_len, const int32_t* length, int B,
                    int n, int32_t* dev_status, void* stream) {
  const int rc = check_fp8(num_blocks, block_size, scale_block, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if ((dt != TS_F32 && dt != TS_BF16) || n <= 0) return TS_ERR_INVALID;
  if (!block_counts(scale_block, d)) return TS_ERR_UNSUPPORTED;
  if (!k || !v || !k_strides || !v_strides || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !start_len)
    return TS_ERR_INVALID;
  const size_t size = dt == TS_BF16 ? 2 : 4;
  ts::Fp8WriteCall c{k, v, dt, {}, {}, k_cache, v_cache, k_scale, v_scale, num_blocks, block_size, scale_block, Hkv, d,
                     block_table, max_blocks, start_len, length, B, n, dev_status};
  for (int i = 0; i < 3; ++i) {
    if (k_strides[i] < 0 || v_strides[i] < 0 || k_strides[i] > (1LL << 40) || v_strides[i] > (1LL << 40)) return TS_ERR_INVALID;
    c.k_stride[i] = k_strides[i];
    c.v_stride[i] = v_strides[i];
  }
  if (reinterpret_cast<uintptr_t>(k) % size != 0 || reinterpret_cast<uintptr_t>(v) % size != 0 || !aligned4_ptr(k_scale) ||
      !aligned4_ptr(v_scale))
    return TS_ERR_INVALID;
  const size_t cache = times(num_blocks, Hkv, block_size, d), scales = times(num_blocks, Hkv, block_size / scale_block);
  if (!outputs_apart({{k_cache, cache, 1}, {v_cache, cache, 1}, {k_scale, scales, 4}, {v_scale, scales, 4}},
                     {{k, extent(k_strides, B, n, Hkv, d), size},
                      {v, extent(v_strides, B, n, Hkv, d), size},
                      {block_table, times(B, max_blocks), 4},
                      {start_len, times(B, 1), 4},
                      {length, times(B, 1), 4}}))
    return TS_ERR_INVALID;
  return ts::kv_write_fp8_launch(c, static_cast<cudaStream_t>(stream));
}

int ts_kv_read_fp8(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int num_blocks,
                   int block_size, int scale_block, int Hkv, int d, const int32_t* block_table, int max_blocks,
                   const int32_t* prefix_len, const int32_t* start_len, int B, int n, void* k, void* v, ts_dtype dt,
                   int32_t* dev_status, void* stream) {
  const int rc = check_fp8(num_blocks, block_size, scale_block, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if ((dt != TS_F32 && dt != TS_BF16) || n <= 0) return TS_ERR_INVALID;
  if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len) return TS_ERR_INVALID;
  const size_t size = dt == TS_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(k) % size != 0 || reinterpret_cast<uintptr_t>(v) % size != 0 || !aligned4_ptr(k_scale) ||
      !aligned4_ptr(v_scale))
    return TS_ERR_INVALID;
  const size_t cache = times(num_blocks, Hkv, block_size, d), scales = times(num_blocks, Hkv, block_size / scale_block);
  const size_t rows = times(B, n, Hkv, d);
  if (!outputs_apart({{k, rows, size}, {v, rows, size}},
                     {{k_cache, cache, 1},
                      {v_cache, cache, 1},
                      {k_scale, scales, 4},
                      {v_scale, scales, 4},
                      {block_table, times(B, max_blocks), 4},
                      {prefix_len, times(B, 1), 4},
                      {start_len, times(B, 1), 4}}))
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  ts::Fp8ReadCall c{k_cache, v_cache, k_scale, v_scale, num_blocks, block_size, scale_block, Hkv, d, block_table, max_blocks,
                    prefix_len, start_len, B, n, k, v, dt, dev_status};
  return ts::kv_read_fp8_launch(c, static_cast<cudaStream_t>(stream), sms);
}

int ts_kv_commit_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int num_blocks, int block_size,
                     int scale_block, int Hkv, int d, const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                     const int32_t* accept_path, const int32_t* accept_len, int B, int m, int32_t* block_table_out,
                     int32_t* prefix_len_out, int32_t* freed_blocks, int32_t* freed_count, int32_t* dev_status, void* stream) {
  const int rc = check_fp8(num_blocks, block_size, scale_block, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (m <= 0) return TS_ERR_INVALID;
  if (m > TS_MAX_NODES || !block_counts(scale_block, d)) return TS_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !accept_path || !accept_len ||
      !block_table_out || !prefix_len_out || !freed_blocks || !freed_count)
    return TS_ERR_INVALID;
  if (!aligned4_ptr(k_scale) || !aligned4_ptr(v_scale)) return TS_ERR_INVALID;
  const size_t cache = times(num_blocks, Hkv, block_size, d), scales = times(num_blocks, Hkv, block_size / scale_block);
  const size_t cells = times(B, max_blocks), rows = B;
  if (!outputs_apart({{k_cache, cache, 1},
                      {v_cache, cache, 1},
                      {k_scale, scales, 4},
                      {v_scale, scales, 4},
                      {block_table_out, cells, 4},
                      {prefix_len_out, rows, 4},
                      {freed_blocks, cells, 4},
                      {freed_count, rows, 4}},
                     {{block_table_out == block_table ? nullptr : block_table, cells, 4},
                      {prefix_len_out == prefix_len ? nullptr : prefix_len, rows, 4},
                      {accept_path, times(B, m), 4},
                      {accept_len, rows, 4}}))
    return TS_ERR_INVALID;
  ts::Fp8CommitCall c{k_cache, v_cache, k_scale, v_scale, num_blocks, block_size, scale_block, Hkv, d, block_table, max_blocks,
                      prefix_len, accept_path, accept_len, B, m, block_table_out, prefix_len_out, freed_blocks, freed_count,
                      dev_status};
  return ts::kv_commit_fp8_launch(c, static_cast<cudaStream_t>(stream));
}

static int check_attention_fp8(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int max_prefix, int block_size) {
  const int rc = ts::check_attention(dt, B, m, Hq, Hkv, d, max_prefix);
  if (rc != TS_OK) return rc;
  if (block_size <= 0) return TS_ERR_INVALID;
  if (max_prefix > (1 << 30)) return TS_ERR_UNSUPPORTED;  // positions and their tiles are counted in 32 bits
  return TS_OK;
}

size_t ts_tree_attention_fp8_workspace(ts_dtype dt, int B, int m, int Hq, int Hkv, int d, int max_prefix, int block_size) {
  if (check_attention_fp8(dt, B, m, Hq, Hkv, d, max_prefix, block_size) != TS_OK) return 0;
  const int sms = ts::device_sm_count();
  return ts::attention_fp8_uses_tc(dt, d, block_size) ? ts::attention_fp8_tc_workspace_bytes(B, m, Hq, Hkv, max_prefix, sms)
                                                      : ts::attention_fp8_simt_workspace_bytes(B, m, Hq, Hkv, d, max_prefix, sms);
}

int ts_tree_attention_fp8(const void* q, ts_dtype dt, const void* k_cache, const void* v_cache, const float* k_scale,
                          const float* v_scale, int num_blocks, int block_size, int scale_block, const int32_t* block_table,
                          int max_blocks, const int32_t* prefix_len, int max_prefix, const uint64_t* mask, int B, int m,
                          int Hq, int Hkv, int d, float scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                          int32_t* dev_status, void* stream) {
  int rc = check_attention_fp8(dt, B, m, Hq, Hkv, d, max_prefix, block_size);
  if (rc != TS_OK) return rc;
  rc = check_fp8(num_blocks, block_size, scale_block, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !prefix_len || !mask || !out) return TS_ERR_INVALID;
  if (!std::isfinite(scale) || !(scale > 0.f)) return TS_ERR_INVALID;
  const size_t size = dt == TS_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(q) % size != 0 || reinterpret_cast<uintptr_t>(out) % size != 0 || !aligned4_ptr(k_scale) ||
      !aligned4_ptr(v_scale))
    return TS_ERR_INVALID;
  const bool tc = ts::attention_fp8_uses_tc(dt, d, block_size);
  if (tc && (!aligned16_ptr(q) || !aligned16_ptr(k_cache) || !aligned16_ptr(v_cache) || !aligned16_ptr(out))) return TS_ERR_INVALID;
  const size_t need = ts_tree_attention_fp8_workspace(dt, B, m, Hq, Hkv, d, max_prefix, block_size);
  if (need > 256 && (!workspace || ws_bytes < need)) return TS_ERR_WORKSPACE;
  if (need > 256 && !aligned16_ptr(workspace)) return TS_ERR_INVALID;
  const size_t rows = times(B, m, Hq), cache = times(num_blocks, Hkv, block_size, d);
  const size_t scales = times(num_blocks, Hkv, block_size / scale_block);
  if (!outputs_apart({{out, rows * d, size}, {lse, rows, 4}, {workspace, need > 256 ? need : 0, 1}},
                     {{q, rows * d, size},
                      {k_cache, cache, 1},
                      {v_cache, cache, 1},
                      {k_scale, scales, 4},
                      {v_scale, scales, 4},
                      {block_table, times(B, max_blocks), 4},
                      {prefix_len, times(B, 1), 4},
                      {mask, times(B, m, (m + 63) / 64), 8}}))
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  ts::Fp8AttnCall a{q, dt, k_cache, v_cache, k_scale, v_scale, num_blocks, block_size, scale_block, block_table, max_blocks,
                    prefix_len, max_prefix, mask, B, m, Hq, Hkv, d, scale, out, lse, workspace, dev_status};
  return tc ? ts::attention_fp8_tc_launch(a, static_cast<cudaStream_t>(stream), sms)
            : ts::attention_fp8_simt_launch(a, static_cast<cudaStream_t>(stream), sms);
}

size_t ts_kv_reserve_workspace(int num_blocks, int block_size, int B, int n) {
  if (num_blocks <= 0 || block_size <= 0 || B <= 0 || n <= 0 || B > TS_MAX_POOL_ROWS) return 0;
  return ts::kv_reserve_workspace_bytes(num_blocks, block_size, B, n);
}

// Both forms of ts_kv_reserve; the caller has checked the cache's sizes.
static int reserve(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int scale_block, int elem_bytes, int num_blocks,
                   int block_size, int Hkv, int d, const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                   const int32_t* refs, int B, int n, const int32_t* freed, int num_freed, int32_t* block_table_out,
                   int32_t* refs_out, int32_t* granted, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (num_blocks > (1 << 28)) return TS_ERR_UNSUPPORTED;
  if (n <= 0 || num_freed < 0 || (num_freed > 0 && !freed)) return TS_ERR_INVALID;
  if (static_cast<long long>(d) * elem_bytes % 4 != 0) return TS_ERR_INVALID;
  if (B > TS_MAX_POOL_ROWS) return TS_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * max_blocks > INT32_MAX) return TS_ERR_UNSUPPORTED;  // requests are counted in 32 bits
  if (!k_cache || !v_cache || !block_table || !prefix_len || !refs || !block_table_out || !refs_out || !granted || !workspace)
    return TS_ERR_INVALID;
  if (!aligned4_ptr(k_cache) || !aligned4_ptr(v_cache) || !aligned16_ptr(workspace)) return TS_ERR_INVALID;
  const size_t need = ts::kv_reserve_workspace_bytes(num_blocks, block_size, B, n);
  if (ws_bytes < need) return TS_ERR_WORKSPACE;
  const size_t cache = times(num_blocks, Hkv, block_size, d), size = elem_bytes, cells = times(B, max_blocks);
  const size_t scales = k_scale ? times(num_blocks, Hkv, block_size / scale_block) : 0;
  if (!outputs_apart({{block_table_out, cells, 4}, {refs_out, times(num_blocks, 1), 4}, {granted, times(B, 1), 4}, {workspace, need, 1}},
                     {{block_table_out == block_table ? nullptr : block_table, cells, 4},
                      {refs_out == refs ? nullptr : refs, times(num_blocks, 1), 4},
                      {prefix_len, times(B, 1), 4},
                      {freed, times(num_freed, 1), 4},
                      {k_cache, cache, size},
                      {v_cache, cache, size},
                      {k_scale, scales, 4},
                      {v_scale, scales, 4}}))
    return TS_ERR_INVALID;
  ts::ReserveCall c{k_cache, v_cache, k_scale, v_scale, scale_block, elem_bytes, num_blocks, block_size, Hkv, d, block_table,
                    max_blocks, prefix_len, refs, B, n, freed, num_freed, block_table_out, refs_out, granted, workspace,
                    dev_status};
  return ts::kv_reserve_launch(c, static_cast<cudaStream_t>(stream));
}

int ts_kv_reserve(void* k_cache, void* v_cache, ts_dtype dt, int num_blocks, int block_size, int Hkv, int d,
                  const int32_t* block_table, int max_blocks, const int32_t* prefix_len, const int32_t* refs,
                  int B, int n, const int32_t* freed, int num_freed, int32_t* block_table_out,
                  int32_t* refs_out, int32_t* granted, void* workspace, size_t ws_bytes, int32_t* dev_status,
                  void* stream) {
  const int rc = check_cache(dt, num_blocks, block_size, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  return reserve(k_cache, v_cache, nullptr, nullptr, 0, dt == TS_BF16 ? 2 : 4, num_blocks, block_size, Hkv, d, block_table,
                 max_blocks, prefix_len, refs, B, n, freed, num_freed, block_table_out, refs_out, granted, workspace, ws_bytes,
                 dev_status, stream);
}

int ts_kv_reserve_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int num_blocks, int block_size,
                      int scale_block, int Hkv, int d, const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                      const int32_t* refs, int B, int n, const int32_t* freed, int num_freed, int32_t* block_table_out,
                      int32_t* refs_out, int32_t* granted, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_fp8(num_blocks, block_size, scale_block, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (!fp8_scales(k_cache, v_cache, k_scale, v_scale, num_blocks, block_size, scale_block, Hkv, d)) return TS_ERR_INVALID;
  return reserve(k_cache, v_cache, k_scale, v_scale, scale_block, 1, num_blocks, block_size, Hkv, d, block_table, max_blocks,
                 prefix_len, refs, B, n, freed, num_freed, block_table_out, refs_out, granted, workspace, ws_bytes, dev_status,
                 stream);
}

int ts_kv_fork(const int32_t* block_table, int max_blocks, const int32_t* prefix_len, const int32_t* refs,
               int num_blocks, int block_size, int B, const int32_t* src, int B_out, int32_t* block_table_out,
               int32_t* prefix_len_out, int32_t* refs_out, int32_t* dev_status, void* stream) {
  if (num_blocks <= 0 || block_size <= 0 || max_blocks <= 0 || B <= 0 || B_out <= 0) return TS_ERR_INVALID;
  if (B > 65535 || B_out > 65535) return TS_ERR_UNSUPPORTED;
  if (!block_table || !prefix_len || !refs || !src || !block_table_out || !prefix_len_out || !refs_out) return TS_ERR_INVALID;
  const size_t rows = B_out, pages = num_blocks;
  if (!outputs_apart({{block_table_out, times(B_out, max_blocks), 4}, {prefix_len_out, rows, 4}, {refs_out, pages, 4}},
                     {{block_table, times(B, max_blocks), 4},
                      {prefix_len, times(B, 1), 4},
                      {refs_out == refs ? nullptr : refs, pages, 4},
                      {src, rows, 4}}))
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  return ts::kv_fork_launch(block_table, max_blocks, prefix_len, refs, num_blocks, block_size, B, src, B_out, block_table_out,
                            prefix_len_out, refs_out, dev_status, static_cast<cudaStream_t>(stream), sms);
}

size_t ts_kv_compact_workspace(int num_blocks) { return num_blocks > 0 ? ts::kv_compact_workspace_bytes(num_blocks) : 0; }

// Both forms of ts_kv_compact; the caller has checked the cache's sizes.  side: smaller buffers of 4-byte words that move
// too, side_words in a page.
static int compact(void* k_cache, void* v_cache, int elem_bytes, void* side0, void* side1, long long side_words, int num_blocks,
                   int block_size, int Hkv, int d, const int32_t* block_table, int max_blocks, const int32_t* refs, int B,
                   int32_t* block_table_out, int32_t* refs_out, int32_t* remap, int32_t* live, void* workspace,
                   size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (static_cast<long long>(d) * elem_bytes % 4 != 0) return TS_ERR_INVALID;
  if (!k_cache || !v_cache || !block_table || !refs || !block_table_out || !refs_out || !remap || !live || !workspace)
    return TS_ERR_INVALID;
  if (!aligned4_ptr(k_cache) || !aligned4_ptr(v_cache) || !aligned16_ptr(workspace)) return TS_ERR_INVALID;
  if (num_blocks > (1 << 28)) return TS_ERR_UNSUPPORTED;
  const size_t need = ts::kv_compact_workspace_bytes(num_blocks);
  if (ws_bytes < need) return TS_ERR_WORKSPACE;
  const size_t cache = times(num_blocks, Hkv, block_size, d), size = elem_bytes, cells = times(B, max_blocks);
  const size_t pages = num_blocks, words = pages * static_cast<size_t>(side_words);
  if (!outputs_apart({{block_table_out, cells, 4}, {refs_out, pages, 4}, {remap, pages, 4}, {live, 1, 4}, {workspace, need, 1}},
                     {{block_table_out == block_table ? nullptr : block_table, cells, 4},
                      {refs_out == refs ? nullptr : refs, pages, 4},
                      {k_cache, cache, size},
                      {v_cache, cache, size},
                      {side0, words, 4},
                      {side1, words, 4}}))
    return TS_ERR_INVALID;
  const int sms = ts::device_sm_count();
  if (sms <= 0) return TS_ERR_CUDA;
  ts::CompactCall c{k_cache, v_cache, {side0, side1}, side_words * 4, num_blocks, block_size, Hkv, d * elem_bytes, block_table,
                    max_blocks, refs, B, block_table_out, refs_out, remap, live, workspace, dev_status};
  return ts::kv_compact_launch(c, static_cast<cudaStream_t>(stream), sms);
}

int ts_kv_compact(void* k_cache, void* v_cache, ts_dtype dt, void* bounds, int num_blocks, int block_size,
                  int Hkv, int d, const int32_t* block_table, int max_blocks, const int32_t* refs, int B,
                  int32_t* block_table_out, int32_t* refs_out, int32_t* remap, int32_t* live, void* workspace,
                  size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_cache(dt, num_blocks, block_size, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (bounds && !aligned16_ptr(bounds)) return TS_ERR_INVALID;
  return compact(k_cache, v_cache, dt == TS_BF16 ? 2 : 4, bounds, nullptr, static_cast<long long>(Hkv) * d, num_blocks, block_size,
                 Hkv, d, block_table, max_blocks, refs, B, block_table_out, refs_out, remap, live, workspace, ws_bytes, dev_status,
                 stream);
}

int ts_kv_compact_fp8(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int num_blocks, int block_size,
                      int scale_block, int Hkv, int d, const int32_t* block_table, int max_blocks, const int32_t* refs, int B,
                      int32_t* block_table_out, int32_t* refs_out, int32_t* remap, int32_t* live, void* workspace,
                      size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_fp8(num_blocks, block_size, scale_block, Hkv, d, max_blocks, B);
  if (rc != TS_OK) return rc;
  if (!fp8_scales(k_cache, v_cache, k_scale, v_scale, num_blocks, block_size, scale_block, Hkv, d)) return TS_ERR_INVALID;
  return compact(k_cache, v_cache, 1, k_scale, v_scale, static_cast<long long>(Hkv) * (block_size / scale_block), num_blocks,
                 block_size, Hkv, d, block_table, max_blocks, refs, B, block_table_out, refs_out, remap, live, workspace, ws_bytes,
                 dev_status, stream);
}

int ts_selftest_bounded_wait(int mode, int32_t* result, int32_t* dev_status, void* stream) {
  if ((mode != 0 && mode != 1) || !result) return TS_ERR_INVALID;
  return ts::selftest_bounded_wait_launch(mode, result, dev_status, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
