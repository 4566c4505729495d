// C ABI of libtreeverify: host-side argument checks, workspace carving and launches.
// Nothing here allocates device memory, synchronises the stream or throws.
#include <math.h>

#include <atomic>

#include <nvtx3/nvToolsExt.h>

#include "tv_kernels.cuh"

using namespace tv;

// Process-wide settings, read at every launch (atomics: another host thread may change
// them while launches are being made).
// SM shares for running the vocab pass and the tree attention concurrently (0 = all SMs)
static std::atomic<int> g_sm_verify{0}, g_sm_attention{0};
// tensor-core attention kernel: 0 automatic, 1 one row tile per CTA, 2 paired row tiles,
// 3 paired row tiles with 64-key KV tiles and double-buffered S, 4 variant 3 on a
// persistent grid
static std::atomic<int> g_attn_variant{0};
// KV splits per tensor-core attention CTA group: 0 automatic, else forced (capped at the
// KV tile count and the cluster limit)
static std::atomic<int> g_attn_splits{0};

namespace tv {
int sm_share_verify() { return g_sm_verify.load(std::memory_order_relaxed); }
int sm_share_attention() { return g_sm_attention.load(std::memory_order_relaxed); }
int attention_variant() { return g_attn_variant.load(std::memory_order_relaxed); }
int attention_splits() { return g_attn_splits.load(std::memory_order_relaxed); }
}  // namespace tv

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_dtype(tv_dtype d) { return d == TV_F32 || d == TV_BF16; }
inline tv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TV_OK : TV_ERR_CUDA; }
inline cudaStream_t st(tv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// One NVTX range per entry point that launches work, named after the entry point, so
// that a profiler's timeline groups each call's kernels.  NVTX is header-only: without an
// attached tool a push or pop is one pointer check.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace

extern "C" {

const char* tv_status_string(int s) {
  switch (s) {
    case TV_OK:
      return "TV_OK";
    case TV_ERR_NULL:
      return "TV_ERR_NULL: a required pointer is NULL";
    case TV_ERR_SHAPE:
      return "TV_ERR_SHAPE: a size is outside the supported range";
    case TV_ERR_DTYPE:
      return "TV_ERR_DTYPE: unsupported dtype";
    case TV_ERR_WORKSPACE:
      return "TV_ERR_WORKSPACE: workspace missing or too small";
    case TV_ERR_ALIGN:
      return "TV_ERR_ALIGN: pointer or stride misaligned";
    case TV_ERR_UNSUPPORTED:
      return "TV_ERR_UNSUPPORTED: combination not implemented";
    case TV_ERR_CUDA:
      return "TV_ERR_CUDA: CUDA call failed while enqueueing";
    case TV_ERR_VALUE:
      return "TV_ERR_VALUE: scalar argument out of range";
    default:
      return "unknown tv_status";
  }
}

int tv_version(void) { return (1 << 16) | 0; }

tv_status tv_philox4x32_10(uint64_t seed, const uint32_t* counters, int n, uint32_t* out, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_philox4x32_10");
  if (n < 0) return TV_ERR_SHAPE;
  if (n > 0 && (!counters || !out)) return TV_ERR_NULL;
  if (!aligned16(counters) || !aligned16(out)) return TV_ERR_ALIGN;
  return cuda_status(launch_philox_words(seed, counters, n, out, st(stream)));
}

tv_status tv_selftest_bounded_wait(int wait_us, int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_selftest_bounded_wait");
  if (!dev_status) return TV_ERR_NULL;
  if (wait_us < 1 || wait_us > 1000000) return TV_ERR_VALUE;
  return cuda_status(launch_wait_selftest((uint64_t)wait_us * 1000ull, dev_status, st(stream)));
}

tv_status tv_set_sm_partition(int verify_sms, int attention_sms) {
  if (verify_sms < 0 || attention_sms < 0) return TV_ERR_VALUE;
  g_sm_verify.store(verify_sms, std::memory_order_relaxed);
  g_sm_attention.store(attention_sms, std::memory_order_relaxed);
  return TV_OK;
}

tv_status tv_set_attention_variant(int variant) {
  if (variant < 0 || variant > 5) return TV_ERR_VALUE;
  g_attn_variant.store(variant, std::memory_order_relaxed);
  return TV_OK;
}

tv_status tv_set_attention_splits(int splits) {
  if (splits < 0 || splits > 8) return TV_ERR_VALUE;
  g_attn_splits.store(splits, std::memory_order_relaxed);
  return TV_OK;
}

tv_status tv_tree_prep(const int32_t* parent, int B, int N, int P, int32_t* depth, int32_t* pos, uint32_t* anc_mask,
                       int32_t* child_off, int32_t* child_idx, int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_tree_prep");
  if (!parent) return TV_ERR_NULL;
  if (B < 1 || N < 1 || N > kMaxNodes || P < 0) return TV_ERR_SHAPE;
  if ((child_off == nullptr) != (child_idx == nullptr)) return TV_ERR_NULL;
  return cuda_status(launch_tree_prep(parent, B, N, P, depth, pos, anc_mask, child_off, child_idx, dev_status,
                                      st(stream)));
}

tv_status tv_prune_tree(const int32_t* parent, const float* conf, int B, int N, int max_children, int depth_limit,
                        int32_t* old_to_new, int32_t* new_parent, int32_t* n_kept, int32_t* new_root,
                        int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_prune_tree");
  if (!parent || !conf || !old_to_new || !new_parent || !n_kept || !new_root) return TV_ERR_NULL;
  if (B < 1 || N < 1 || N > kMaxNodes) return TV_ERR_SHAPE;
  if (max_children < 1 || depth_limit < 1) return TV_ERR_VALUE;
  return cuda_status(launch_prune(parent, conf, B, N, max_children, depth_limit, old_to_new, new_parent, n_kept,
                                  new_root, dev_status, st(stream)));
}

size_t tv_tree_attention_workspace_size(int B, int Hq, int Hkv, int D, int P, int N, tv_dtype dtype) {
  if (B < 1 || Hq < 1 || Hkv < 1 || D < 1 || P < 0 || N < 1) return 0;
  AttnPlan p = attn_plan(B, Hq, Hkv, D, P, N, dtype);
  return p.tc ? p.total : 0;
}

tv_status tv_tree_attention(const void* q, const void* k_cache, const void* v_cache, void* out,
                            const int32_t* parent, int B, int Hq, int Hkv, int D, int P, int N, int kv_stride_tokens,
                            float scale, tv_dtype dtype, void* workspace, size_t ws_bytes, int32_t* dev_status,
                            tv_stream_t stream) {
  NvtxRange nvtx_range("tv_tree_attention");
  if (!q || !k_cache || !v_cache || !out || !parent) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || N < 1 || N > kMaxNodes || P < 0) return TV_ERR_SHAPE;
  if (D < 32 || D > 256 || D % 32) return TV_ERR_SHAPE;
  if ((long long)kv_stride_tokens < (long long)P + N) return TV_ERR_SHAPE;
  if ((long long)B * Hkv > 65535LL * 65535LL) return TV_ERR_SHAPE;
  if (!(scale >= 0.f) || isinf(scale)) return TV_ERR_VALUE;
  if (scale == 0.f) scale = 1.f / sqrtf((float)D);
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return TV_ERR_ALIGN;
  AttnPlan p = attn_plan(B, Hq, Hkv, D, P, N, dtype);
  if (p.tc) {
    if (B > 65535 || Hkv > 65535) return TV_ERR_SHAPE;
    if (workspace && !aligned16(workspace)) return TV_ERR_ALIGN;
    return cuda_status(launch_attn_tc(q, k_cache, v_cache, out, parent, B, Hq, Hkv, D, P, N, kv_stride_tokens, scale,
                                      p, reinterpret_cast<char*>(workspace), ws_bytes, dev_status, st(stream)));
  }
  if ((long long)B * Hq * N / 4 + 1 > 0x7fffffffLL) return TV_ERR_SHAPE;
  return cuda_status(launch_attn_simt(q, k_cache, v_cache, out, parent, B, Hq, Hkv, D, P, N, kv_stride_tokens, scale,
                                      dtype, dev_status, st(stream)));
}

tv_status tv_tree_attention_plan(int B, int Hq, int Hkv, int D, int P, int N, tv_dtype dtype, int* kernel,
                                 int* splits) {
  if (!kernel || !splits) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || N < 1 || N > kMaxNodes || P < 0) return TV_ERR_SHAPE;
  AttnPlan p = attn_plan(B, Hq, Hkv, D, P, N, dtype);
  if (!p.tc) {
    *kernel = 0;
    *splits = 1;
    return TV_OK;
  }
  attn_tc_choice(B, Hkv, D, P, N, p, kernel, splits);
  return TV_OK;
}

size_t tv_verify_workspace_size(int B, int N, int V, tv_dtype, int sampling) {
  if (B < 1 || N < 1 || V < 1) return 0;
  return verify_ws_layout(B, N, V, sampling ? 1 : 0, nullptr);
}

static tv_status verify_common_checks(const void* logits, const int32_t* parent, const int32_t* tokens, int B, int N,
                                      int V, tv_dtype dtype, void* ws, size_t ws_bytes, int sampling) {
  if (!logits || !parent || !tokens) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (B < 1 || N < 1 || N > kMaxNodes || V < 1) return TV_ERR_SHAPE;
  const long long rows = (long long)B * N;
  if (rows > kMaxVerifyRows) return TV_ERR_SHAPE;
  if ((long long)N * V > 0x7fffffffLL) return TV_ERR_SHAPE;
  if (!ws || ws_bytes < verify_ws_layout(B, N, V, sampling, nullptr)) return TV_ERR_WORKSPACE;
  if (!aligned16(ws)) return TV_ERR_ALIGN;
  return TV_OK;
}

tv_status tv_verify_greedy(const void* logits, const int32_t* parent, const int32_t* tokens, int B, int N, int V,
                           tv_dtype dtype, int32_t* accepted_nodes, int32_t* accept_len, int32_t* bonus_token,
                           float* p_draft, float* row_lse, int32_t* row_argmax, void* workspace, size_t ws_bytes,
                           int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_verify_greedy");
  if (!accepted_nodes || !accept_len || !bonus_token) return TV_ERR_NULL;
  tv_status s = verify_common_checks(logits, parent, tokens, B, N, V, dtype, workspace, ws_bytes, 0);
  if (s != TV_OK) return s;
  VerifyWs w;
  verify_ws_layout(B, N, V, 0, &w);
  return cuda_status(launch_vocab_pass(logits, nullptr, parent, tokens, B, N, V, dtype, 1.0f,
                                       reinterpret_cast<char*>(workspace), w, accepted_nodes, accept_len, bonus_token,
                                       p_draft, nullptr, row_lse, row_argmax, nullptr, dev_status, 0,
                                       st(stream)));
}

tv_status tv_vocab_stats(const void* logits, const void* draft_logits, const int32_t* parent,
                         const int32_t* tokens, int B, int N, int V, float temperature, tv_dtype dtype,
                         float* row_lse, int32_t* row_argmax, float* p_draft, float* draft_row_lse, float* q_draft,
                         void* workspace, size_t ws_bytes, int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_vocab_stats");
  if (!draft_logits && (draft_row_lse || q_draft)) return TV_ERR_NULL;
  if (!(temperature > 0.f) || isinf(temperature)) return TV_ERR_VALUE;
  const int two = draft_logits ? 1 : 0;
  tv_status s = verify_common_checks(logits, parent, tokens, B, N, V, dtype, workspace, ws_bytes, two);
  if (s != TV_OK) return s;
  VerifyWs w;
  verify_ws_layout(B, N, V, two, &w);
  return cuda_status(launch_vocab_pass(logits, draft_logits, parent, tokens, B, N, V, dtype, temperature,
                                       reinterpret_cast<char*>(workspace), w, nullptr, nullptr, nullptr, p_draft,
                                       q_draft, row_lse, row_argmax, draft_row_lse, dev_status, two, st(stream)));
}

tv_status tv_verify_sample(const void* target_logits, const void* draft_logits, const int32_t* parent,
                           const int32_t* tokens, int B, int N, int V, float temperature, uint64_t seed,
                           uint64_t round, tv_dtype dtype, int32_t* accepted_nodes, int32_t* accept_len,
                           int32_t* out_token, float* p_draft, float* q_draft, void* workspace, size_t ws_bytes,
                           int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_verify_sample");
  if (!draft_logits || !accepted_nodes || !accept_len || !out_token) return TV_ERR_NULL;
  if (!(temperature > 0.f) || isinf(temperature)) return TV_ERR_VALUE;
  tv_status s = verify_common_checks(target_logits, parent, tokens, B, N, V, dtype, workspace, ws_bytes, 1);
  if (s != TV_OK) return s;
  VerifyWs w;
  verify_ws_layout(B, N, V, 1, &w);
  char* ws = reinterpret_cast<char*>(workspace);
  cudaError_t e = launch_vocab_pass(target_logits, draft_logits, parent, tokens, B, N, V, dtype, temperature, ws, w,
                                    nullptr, nullptr, nullptr, p_draft, q_draft, nullptr, nullptr, nullptr,
                                    dev_status, 1, st(stream));
  if (e != cudaSuccess) return TV_ERR_CUDA;
  return cuda_status(launch_sample_walk(target_logits, draft_logits, parent, tokens, B, N, V, dtype, temperature,
                                        seed, round, ws, w, accepted_nodes, accept_len, out_token, dev_status,
                                        st(stream)));
}

tv_status tv_commit_accepted_kv(void* k_cache, void* v_cache, const int32_t* accepted_nodes,
                                const int32_t* accept_len, int B, int Hkv, int D, int P, int N, int kv_stride_tokens,
                                tv_dtype dtype, int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_commit_accepted_kv");
  if (!k_cache || !v_cache || !accepted_nodes || !accept_len) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (B < 1 || Hkv < 1 || D < 1 || P < 0 || N < 1 || N > kMaxNodes) return TV_ERR_SHAPE;
  if ((long long)kv_stride_tokens < (long long)P + N) return TV_ERR_SHAPE;
  const long long row_bytes = (long long)D * (dtype == TV_BF16 ? 2 : 4);
  if (row_bytes % 16) return TV_ERR_ALIGN;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return TV_ERR_ALIGN;
  if ((long long)B * Hkv * 2 * (row_bytes / 16) > 0x7fffffffLL * 256) return TV_ERR_SHAPE;
  return cuda_status(launch_kv_commit(k_cache, v_cache, accepted_nodes, accept_len, B, Hkv, D, P, N,
                                      kv_stride_tokens, dtype, dev_status, st(stream)));
}

tv_status tv_frontier_topw(const float* scores, const int32_t* count, int B, int C, int W, int32_t* out_idx,
                           int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_frontier_topw");
  if (!scores || !count || !out_idx) return TV_ERR_NULL;
  if (B < 1 || C < 1 || C > 4096 || W < 1 || W > C) return TV_ERR_SHAPE;
  return cuda_status(launch_frontier_topw(scores, count, B, C, W, out_idx, dev_status, st(stream)));
}

size_t tv_expand_workspace_size(int R, int V, int m) { return expand_ws_bytes(R, V, m); }

tv_status tv_expand_children(const void* draft_logits, const float* parent_score, int R, int V, int m,
                             float temperature, tv_dtype dtype, int32_t* child_token, float* child_p,
                             float* child_score, void* workspace, size_t ws_bytes, int32_t* dev_status,
                             tv_stream_t stream) {
  NvtxRange nvtx_range("tv_expand_children");
  if (!draft_logits || !parent_score || !child_token || !child_p || !child_score) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (R < 1 || V < 1 || m < 1 || m > 32) return TV_ERR_SHAPE;
  if ((long long)R * 32 > 0x7fffffffLL) return TV_ERR_SHAPE;
  if (!(temperature > 0.f) || isinf(temperature)) return TV_ERR_VALUE;
  if (!workspace || ws_bytes < expand_ws_bytes(R, V, m)) return TV_ERR_WORKSPACE;
  if (!aligned16(workspace)) return TV_ERR_ALIGN;
  return cuda_status(launch_expand(draft_logits, parent_score, R, V, m, temperature, dtype, child_token, child_p,
                                   child_score, reinterpret_cast<char*>(workspace), dev_status, st(stream)));
}

size_t tv_select_workspace_size(int B, int d, int K, int budget) { return select_ws_bytes(B, d, K, budget); }

tv_status tv_select_subtree(const float* marg, const int32_t* pool_tokens, int B, int d, int K, int budget,
                            const int32_t* root_token, int32_t* parent, int32_t* tokens, int32_t* depth, float* score,
                            int32_t* n_nodes, void* workspace, size_t ws_bytes, int32_t* dev_status,
                            tv_stream_t stream) {
  NvtxRange nvtx_range("tv_select_subtree");
  if (!marg || !pool_tokens || !parent || !tokens || !depth || !score) return TV_ERR_NULL;
  if (B < 1 || d < 1 || d > kMaxDepth || K < 1 || K > kMaxRank || budget < 1 || budget > kMaxBudget)
    return TV_ERR_SHAPE;
  if (ws_bytes < select_ws_bytes(B, d, K, budget)) return TV_ERR_WORKSPACE;
  return cuda_status(launch_select(marg, pool_tokens, B, d, K, budget, root_token, parent, tokens, depth, score,
                                   n_nodes, reinterpret_cast<char*>(workspace), dev_status, 0.f, 0.f, st(stream)));
}

tv_status tv_select_subtree_adaptive(const float* marg, const int32_t* pool_tokens, int B, int d, int K, int budget,
                                     float cost_base, float cost_per_row, const int32_t* root_token, int32_t* parent,
                                     int32_t* tokens, int32_t* depth, float* score, int32_t* n_nodes,
                                     void* workspace, size_t ws_bytes, int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_select_subtree_adaptive");
  if (!marg || !pool_tokens || !parent || !tokens || !depth || !score || !n_nodes) return TV_ERR_NULL;
  if (B < 1 || d < 1 || d > kMaxDepth || K < 1 || K > kMaxRank || budget < 1 || budget > kMaxBudget)
    return TV_ERR_SHAPE;
  if (!(cost_base >= 0.f) || isinf(cost_base) || !(cost_per_row > 0.f) || isinf(cost_per_row)) return TV_ERR_VALUE;
  if (ws_bytes < select_ws_bytes(B, d, K, budget)) return TV_ERR_WORKSPACE;
  return cuda_status(launch_select(marg, pool_tokens, B, d, K, budget, root_token, parent, tokens, depth, score,
                                   n_nodes, reinterpret_cast<char*>(workspace), dev_status, cost_base, cost_per_row,
                                   st(stream)));
}

tv_status tv_rotary_frequencies(int rot_dim, double base, int scaling, const double* params, uint64_t* freq,
                                float* amplitude) {
  if (!freq || !amplitude) return TV_ERR_NULL;
  if (rot_dim < 2 || rot_dim > kMaxRotaryDim || rot_dim % 2) return TV_ERR_SHAPE;
  if (!(base > 1.0) || isinf(base)) return TV_ERR_VALUE;
  if (scaling < TV_ROPE_NONE || scaling > TV_ROPE_YARN) return TV_ERR_VALUE;
  if (scaling != TV_ROPE_NONE) {
    if (!params) return TV_ERR_NULL;
    const int n = scaling >= TV_ROPE_BANDED ? 4 : 1;
    for (int i = 0; i < n; ++i)
      if (!isfinite(params[i])) return TV_ERR_VALUE;
    if (params[0] < 1.0) return TV_ERR_VALUE;
    if (scaling == TV_ROPE_BASE && rot_dim < 4) return TV_ERR_SHAPE;
    if (scaling == TV_ROPE_BANDED && (!(params[2] > params[1]) || !(params[3] > 0.0))) return TV_ERR_VALUE;
    if (scaling == TV_ROPE_YARN && (!(params[1] > 0.0) || !(params[3] > 0.0) || params[2] < params[3]))
      return TV_ERR_VALUE;
  }
  rotary_frequencies(rot_dim, base, scaling, params, freq, amplitude);
  return TV_OK;
}

// rows: a pointer aligned to its element
static bool rows_aligned(const tv_rows* r, tv_dtype dtype) {
  return reinterpret_cast<uintptr_t>(r->data) % (dtype == TV_BF16 ? 2 : 4) == 0;
}
static void rows_arg(RotaryArgs* a, int part, const tv_rows* r) {
  a->src[part] = r->data;
  a->sb[part] = r->batch_stride;
  a->sh[part] = r->head_stride;
  a->sn[part] = r->row_stride;
}
static tv_status rope_checks(const tv_rope* rope, int D) {
  if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 2) return TV_ERR_SHAPE;
  if (rope->rot_dim > 0 && !rope->freq) return TV_ERR_NULL;
  if (!isfinite(rope->amplitude)) return TV_ERR_VALUE;
  return TV_OK;
}

tv_status tv_rotary(const tv_rows* x, void* out, const int32_t* pos, const int32_t* pos_base, const tv_rope* rope,
                    int B, int H, int N, int D, tv_dtype dtype, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_rotary");
  if (!x || !x->data || !out || !pos || !rope) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (B < 1 || H < 1 || H > kMaxRotaryHeads || N < 1 || D < 1 || D > kMaxRotaryDim) return TV_ERR_SHAPE;
  if ((long long)B * N > kMaxRotaryRows) return TV_ERR_SHAPE;
  const tv_status s = rope_checks(rope, D);
  if (s != TV_OK) return s;
  if (!rows_aligned(x, dtype) || reinterpret_cast<uintptr_t>(out) % (dtype == TV_BF16 ? 2 : 4)) return TV_ERR_ALIGN;
  RotaryArgs a{};
  rows_arg(&a, 0, x);
  a.q_out = out;
  a.pos = pos;
  a.base = pos_base;
  a.freq = rope->freq;
  a.amplitude = rope->amplitude;
  a.B = B, a.Hq = H, a.N = N, a.D = D, a.rot = rope->rot_dim, a.interleaved = rope->interleaved != 0;
  return cuda_status(launch_rotary(a, dtype, st(stream)));
}

static bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

static int log2_exact(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// The checks that every call over a paged cache shares.
static tv_status paged_checks(const tv_paged_kv* kv, int B, int Hkv, int N, int D, tv_dtype dtype) {
  if (!kv || !kv->k || !kv->v || !kv->page_table || !kv->prefix_len) return TV_ERR_NULL;
  if (!valid_dtype(dtype)) return TV_ERR_DTYPE;
  if (B < 1 || Hkv < 1 || Hkv > kMaxRotaryHeads || N < 1 || D < 1 || D > kMaxRotaryDim) return TV_ERR_SHAPE;
  const int ps = kv->page_size;
  if (ps < 8 || ps > 1024 || (ps & (ps - 1)) || kv->num_pages < 1 || kv->max_pages < 1) return TV_ERR_SHAPE;
  if ((long long)kv->max_pages * ps > (1LL << 30) || (long long)kv->num_pages * Hkv > 0x7fffffffLL)
    return TV_ERR_SHAPE;
  if (!aligned16(kv->k) || !aligned16(kv->v) || (long long)D * (dtype == TV_BF16 ? 2 : 4) % 16) return TV_ERR_ALIGN;
  return TV_OK;
}

tv_status tv_append_kv_paged(const tv_rows* k, const tv_rows* v, const tv_paged_kv* kv, const int32_t* depth,
                             const int32_t* n_rows, const tv_rope* rope, const tv_rows* q, void* q_out, int B, int Hq,
                             int Hkv, int N, int D, tv_dtype dtype, int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_append_kv_paged");
  if (!k || !k->data || !v || !v->data) return TV_ERR_NULL;
  if (q && (!q->data || !q_out || !rope)) return TV_ERR_NULL;
  tv_status s = paged_checks(kv, B, Hkv, N, D, dtype);
  if (s != TV_OK) return s;
  if (q && (Hq < 1 || Hq > kMaxRotaryHeads)) return TV_ERR_SHAPE;
  if ((long long)B * N > kMaxRotaryRows) return TV_ERR_SHAPE;
  if (rope) {
    s = rope_checks(rope, D);
    if (s != TV_OK) return s;
  }
  if (!rows_aligned(k, dtype) || !rows_aligned(v, dtype)) return TV_ERR_ALIGN;
  if (q && (!rows_aligned(q, dtype) || reinterpret_cast<uintptr_t>(q_out) % (dtype == TV_BF16 ? 2 : 4)))
    return TV_ERR_ALIGN;
  RotaryArgs a{};
  if (q) rows_arg(&a, 0, q);
  rows_arg(&a, 1, k);
  rows_arg(&a, 2, v);
  a.q_out = q_out;
  a.k_cache = kv->k;
  a.v_cache = kv->v;
  a.pos = depth;
  a.base = kv->prefix_len;
  a.n_rows = n_rows;
  a.table = kv->page_table;
  a.freq = rope ? rope->freq : nullptr;
  a.amplitude = rope ? rope->amplitude : 1.f;
  a.B = B, a.Hq = q ? Hq : 0, a.Hkv = Hkv, a.N = N, a.D = D;
  a.rot = rope ? rope->rot_dim : 0, a.interleaved = rope && rope->interleaved != 0;
  a.num_pages = kv->num_pages, a.page_shift = log2_exact(kv->page_size), a.max_pages = kv->max_pages;
  a.dev_status = dev_status;
  return cuda_status(launch_rotary(a, dtype, st(stream)));
}

static bool paged_attn_shape(int B, int Hq, int Hkv, int N, int D) {
  return B >= 1 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && N >= 1 && N <= kMaxChunk && D >= 32 && D <= 256 &&
         D % 32 == 0 && (long long)(Hq / Hkv) * N < (1 << 24);
}

size_t tv_paged_attention_workspace_size(int B, int Hq, int Hkv, int D, int N, int page_size, int max_pages,
                                         tv_dtype dtype) {
  if (!paged_attn_shape(B, Hq, Hkv, N, D) || page_size < 8 || max_pages < 1 || !valid_dtype(dtype)) return 0;
  return paged_attn_ws(B, Hq, Hkv, D, N, dtype, paged_grid_sms()).bytes;
}

tv_status tv_paged_attention(const void* q, void* out, const tv_paged_kv* kv, const int32_t* parent,
                             const int32_t* n_rows, int B, int Hq, int Hkv, int N, int D, float scale, float softcap,
                             int window, tv_dtype dtype, void* workspace, size_t ws_bytes, int32_t* dev_status,
                             tv_stream_t stream) {
  NvtxRange nvtx_range("tv_paged_attention");
  if (!q || !out) return TV_ERR_NULL;
  const tv_status s = paged_checks(kv, B, Hkv, N, D, dtype);
  if (s != TV_OK) return s;
  if (!paged_attn_shape(B, Hq, Hkv, N, D) || (parent && N > kMaxNodes)) return TV_ERR_SHAPE;
  if (!(scale >= 0.f) || isinf(scale) || !(softcap >= 0.f) || isinf(softcap) || window < 0) return TV_ERR_VALUE;
  if (scale == 0.f) scale = 1.f / sqrtf((float)D);
  if (softcap > 0.f && isinf(4.f * scale / softcap)) return TV_ERR_VALUE;
  if (!aligned16(q) || !aligned16(out)) return TV_ERR_ALIGN;
  const int sms = paged_grid_sms();  // read once: the schedule and its workspace go by it
  const size_t need = paged_attn_ws(B, Hq, Hkv, D, N, dtype, sms).need;
  if (need && (!workspace || ws_bytes < need)) return TV_ERR_WORKSPACE;
  if (!aligned16(workspace)) return TV_ERR_ALIGN;
  const size_t rows_bytes = (size_t)B * Hq * N * D * (dtype == TV_BF16 ? 2 : 4);
  if (overlap(q, rows_bytes, out, rows_bytes)) return TV_ERR_VALUE;
  PagedAttn a{};
  a.q = q, a.out = out, a.k = kv->k, a.v = kv->v;
  a.table = kv->page_table, a.prefix_len = kv->prefix_len, a.parent = parent, a.n_rows = n_rows;
  a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.D = D, a.N = N;
  a.num_pages = kv->num_pages, a.page_shift = log2_exact(kv->page_size), a.max_pages = kv->max_pages;
  a.scale = scale;
  a.cap = softcap;
  a.window = window;
  a.sms = sms;
  a.dev_status = dev_status;
  return cuda_status(launch_paged_attn(a, dtype, reinterpret_cast<char*>(workspace), st(stream)));
}

tv_status tv_commit_accepted_kv_paged(const tv_paged_kv* kv, const int32_t* accepted_nodes, const int32_t* accept_len,
                                      int32_t* new_len, int B, int Hkv, int N, int D, tv_dtype dtype,
                                      int32_t* dev_status, tv_stream_t stream) {
  NvtxRange nvtx_range("tv_commit_accepted_kv_paged");
  if (!accepted_nodes || !accept_len) return TV_ERR_NULL;
  const tv_status s = paged_checks(kv, B, Hkv, N, D, dtype);
  if (s != TV_OK) return s;
  if (N > kMaxNodes || B > 65535) return TV_ERR_SHAPE;
  // a sequence's CTAs read these while its first one writes new_len
  const size_t b4 = (size_t)B * 4;
  if (new_len && (overlap(new_len, b4, kv->prefix_len, b4) || overlap(new_len, b4, accept_len, b4) ||
                  overlap(new_len, b4, accepted_nodes, b4 * N) || overlap(new_len, b4, kv->page_table, b4 * kv->max_pages)))
    return TV_ERR_VALUE;
  return cuda_status(launch_kv_commit_paged(kv->k, kv->v, kv->page_table, kv->prefix_len, accepted_nodes, accept_len,
                                            new_len, B, Hkv, D, N, kv->num_pages, log2_exact(kv->page_size),
                                            kv->max_pages, dtype, dev_status, st(stream)));
}

}  // extern "C"
