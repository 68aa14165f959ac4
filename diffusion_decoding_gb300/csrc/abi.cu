// C ABI of the decode step: argument validation, workspace layout and kernel launches.
// Every entry point validates on the host first and launches nothing when it returns an error.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

namespace {

// One NVTX range per entry point, named after it, spanning the host-side work of the call
// (validation and kernel launches; the kernels themselves run later on the stream).  Free when
// no profiler is attached.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

thread_local char g_err[512];

dllm_status fail(dllm_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

dllm_status ok() {
  g_err[0] = '\0';
  return DLLM_OK;
}

dllm_status cuda_fail(cudaError_t e, const char* where) {
  return fail(DLLM_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
  return n > 0 ? n : 1;
}

dllm_status check_shape(const dllm_shape* sh) {
  if (!sh) return fail(DLLM_ERR_INVALID_ARG, "shape is null");
  if (sh->B < 1 || sh->L < 1 || sh->V < 1)
    return fail(DLLM_ERR_INVALID_ARG, "B, L and V must be positive (B=%d L=%d V=%d)", sh->B,
                sh->L, sh->V);
  if (sh->dtype != DLLM_F32 && sh->dtype != DLLM_BF16)
    return fail(DLLM_ERR_UNSUPPORTED, "dtype %d is not fp32 (0) or bf16 (1)", sh->dtype);
  if (sh->L > dllm::kMaxL) return fail(DLLM_ERR_UNSUPPORTED, "L=%d exceeds %d", sh->L, dllm::kMaxL);
  if (static_cast<int64_t>(sh->B) * sh->L > (int64_t{1} << 20))
    return fail(DLLM_ERR_UNSUPPORTED, "B*L=%lld exceeds 2^20",
                static_cast<long long>(sh->B) * sh->L);
  if (sh->row_stride < sh->V)
    return fail(DLLM_ERR_INVALID_ARG, "row_stride %lld < V %d",
                static_cast<long long>(sh->row_stride), sh->V);
  return DLLM_OK;
}

dllm_status check_ws(const void* ws) {
  if (!ws) return fail(DLLM_ERR_INVALID_ARG, "workspace is null");
  if (!aligned(ws, 256)) return fail(DLLM_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return DLLM_OK;
}

dllm_status check_stats(const dllm_stats* st) {
  if (!st || !st->row_max || !st->lse || !st->conf || !st->argmax)
    return fail(DLLM_ERR_INVALID_ARG, "stats or one of its arrays is null");
  return DLLM_OK;
}

dllm_status check_state(const dllm_block_state* s) {
  if (!s || !s->masked || !s->tokens || !s->committed_now || !s->n_commit || !s->eos_hit)
    return fail(DLLM_ERR_INVALID_ARG, "block state or one of its arrays is null");
  return DLLM_OK;
}

// Logits for the statistics and commit calls: aligned to their element size (rows that are
// not 16-byte aligned take the scalar-load path of the statistics kernel).
dllm_status check_logits(const void* logits, const dllm_shape* sh) {
  if (!aligned(logits, sh->dtype == DLLM_BF16 ? 2 : 4))
    return fail(DLLM_ERR_INVALID_ARG, "logits must be aligned to the element size");
  return DLLM_OK;
}

// Rows the single-read smoothing kernels can copy whole (16-byte aligned rows, V a multiple of
// 8); other layouts take the element-wise path.
bool rows_vector_aligned(const void* logits, const dllm_shape* sh) {
  const int es = sh->dtype == DLLM_BF16 ? 2 : 4;
  return aligned(logits, 16) && (sh->row_stride * es) % 16 == 0 && sh->V % 8 == 0;
}

dllm::CommitArgs threshold_args(float tau, int32_t eos_id) {
  dllm::CommitArgs ca{};
  ca.mode = dllm::kThreshold;
  ca.tau = tau;
  ca.eos_id = eos_id;
  return ca;
}

#define DLLM_TRY(x)                 \
  do {                              \
    dllm_status s_ = (x);           \
    if (s_ != DLLM_OK) return s_;   \
  } while (0)

// The graph `stream` is capturing (with its current capture dependencies when asked for);
// DLLM_ERR_INVALID_ARG when the stream is not capturing.
dllm_status capturing_graph(dllm_stream_t stream, cudaGraph_t* graph, const cudaGraphNode_t** deps,
                            size_t* n_deps, const char* name) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(stream), &cs, nullptr,
                                           graph, deps, nullptr, n_deps);
  if (e != cudaSuccess) return cuda_fail(e, name);
  if (cs != cudaStreamCaptureStatusActive)
    return fail(DLLM_ERR_INVALID_ARG, "%s: stream is not capturing a graph", name);
  return DLLM_OK;
}

// Shared body of the three commit entry points.
dllm_status commit_common(const void* logits, const dllm_shape* shape, const dllm_stats* stats,
                          const dllm_block_state* state, const dllm::CommitArgs& ca, void* ws,
                          dllm_stream_t stream, const char* name) {
  DLLM_TRY(check_shape(shape));
  DLLM_TRY(check_stats(stats));
  DLLM_TRY(check_state(state));
  cudaError_t e;
  if (logits) {
    DLLM_TRY(check_logits(logits, shape));
    DLLM_TRY(check_ws(ws));
    const dllm::StatsWs w = dllm::stats_ws_layout(ws, shape->B, shape->L, shape->V);
    e = dllm::launch_stats_commit(logits, *shape, nullptr, *stats, state, ca, w, sm_count(),
                                  reinterpret_cast<cudaStream_t>(stream));
  } else {
    e = dllm::launch_commit_only(*shape, *stats, *state, ca,
                                 reinterpret_cast<cudaStream_t>(stream));
  }
  if (e != cudaSuccess) return cuda_fail(e, name);
  return ok();
}

// Rows of heads: pointer, dtype and alignment to the element size.
dllm_status check_heads(const dllm_heads* h, const char* what) {
  if (!h || !h->data) return fail(DLLM_ERR_INVALID_ARG, "%s or its data is null", what);
  if (h->dtype != DLLM_F32 && h->dtype != DLLM_BF16)
    return fail(DLLM_ERR_UNSUPPORTED, "%s: dtype %d is not fp32 (0) or bf16 (1)", what, h->dtype);
  if (h->heads < 1 || h->heads > 65536)
    return fail(DLLM_ERR_INVALID_ARG, "%s: heads=%d outside [1, 65536]", what, h->heads);
  if (!aligned(h->data, h->dtype == DLLM_BF16 ? 2 : 4))
    return fail(DLLM_ERR_INVALID_ARG, "%s must be aligned to the element size", what);
  return DLLM_OK;
}

dllm_status check_tokens(int32_t B, int32_t n) {
  if (B < 1 || n < 1) return fail(DLLM_ERR_INVALID_ARG, "need B, n >= 1 (B=%d n=%d)", B, n);
  if (static_cast<int64_t>(B) * n > (int64_t{1} << 20))
    return fail(DLLM_ERR_UNSUPPORTED, "B*n=%lld exceeds 2^20", static_cast<long long>(B) * n);
  return DLLM_OK;
}

dllm_status check_cache(const dllm_kv4_cache* c) {
  if (!c || !c->k_codes || !c->k_params || !c->v_codes || !c->v_params || !c->page_table)
    return fail(DLLM_ERR_INVALID_ARG, "cache or one of its arrays is null");
  if (c->pages < 1 || c->heads < 1 || c->table_stride < 1)
    return fail(DLLM_ERR_INVALID_ARG, "need pages, heads, table_stride >= 1 (%d, %d, %d)", c->pages,
                c->heads, c->table_stride);
  if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 != 0)
    return fail(DLLM_ERR_UNSUPPORTED, "page_size=%d is not a multiple of 16 in [16, 65536]",
                c->page_size);
  if (c->head_dim < 32 || c->head_dim > 512 || c->head_dim % 32 != 0)
    return fail(DLLM_ERR_UNSUPPORTED, "head_dim=%d is not a multiple of 32 in [32, 512]",
                c->head_dim);
  if (c->heads > 4096) return fail(DLLM_ERR_UNSUPPORTED, "heads=%d exceeds 4096", c->heads);
  if (static_cast<int64_t>(c->table_stride) * c->page_size >= (int64_t{1} << 31))
    return fail(DLLM_ERR_UNSUPPORTED, "table_stride * page_size exceeds 2^31 - 1");
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_params, 16) ||
      !aligned(c->v_params, 16) || !aligned(c->page_table, 4))
    return fail(DLLM_ERR_INVALID_ARG, "codes and params must be 16-byte, page_table 4-byte aligned");
  return DLLM_OK;
}

// Shared checks of the cache's write and read.
dllm_status check_cache_rows(const dllm_kv4_cache* cache, const dllm_heads* k, const dllm_heads* v,
                             int32_t B, int32_t n) {
  DLLM_TRY(check_cache(cache));
  DLLM_TRY(check_heads(k, "k"));
  DLLM_TRY(check_heads(v, "v"));
  DLLM_TRY(check_tokens(B, n));
  if (k->dtype != v->dtype) return fail(DLLM_ERR_INVALID_ARG, "k and v differ in dtype");
  if (k->heads != cache->heads || v->heads != cache->heads)
    return fail(DLLM_ERR_INVALID_ARG, "k has %d heads and v %d, the cache %d", k->heads, v->heads,
                cache->heads);
  return DLLM_OK;
}

dllm_status check_attention(const dllm_kv4_cache* cache, int32_t B, int32_t n, int32_t q_heads,
                            int32_t max_len) {
  DLLM_TRY(check_cache(cache));
  DLLM_TRY(check_tokens(B, n));
  if (cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 192 &&
      cache->head_dim != 256)
    return fail(DLLM_ERR_UNSUPPORTED, "head_dim=%d is not 64, 128, 192 or 256", cache->head_dim);
  if (q_heads < 1 || q_heads > 65536 || q_heads % cache->heads != 0)
    return fail(DLLM_ERR_INVALID_ARG, "%d query heads are no multiple of the cache's %d", q_heads,
                cache->heads);
  if (max_len < 0 ||
      max_len > static_cast<int64_t>(cache->table_stride) * cache->page_size)
    return fail(DLLM_ERR_INVALID_ARG, "max_len=%d outside [0, table_stride * page_size]", max_len);
  if (max_len > (1 << 30)) return fail(DLLM_ERR_UNSUPPORTED, "max_len=%d exceeds 2^30", max_len);
  if (static_cast<int64_t>(B) * n * q_heads > (int64_t{1} << 30))
    return fail(DLLM_ERR_UNSUPPORTED, "B * n * heads exceeds 2^30");
  return DLLM_OK;
}

// What a call says of its queries and what they see, checked before.
dllm::AttnParams attention_params(const dllm_heads* q, const dllm_kv4_cache* cache, const int32_t* lens,
                                  int32_t max_len, const uint8_t* key_mask, int64_t mask_stride,
                                  float scale, int32_t causal, int32_t B, int32_t n) {
  dllm::AttnParams p{};
  p.q = static_cast<const uint16_t*>(q->data);
  p.qb = q->batch_stride, p.qt = q->token_stride, p.qh = q->head_stride;
  p.k_codes = cache->k_codes, p.k_params = cache->k_params;
  p.v_codes = cache->v_codes, p.v_params = cache->v_params;
  p.table = cache->page_table;
  p.table_stride = cache->table_stride;
  p.pages = cache->pages;
  p.page_size = cache->page_size;
  p.heads = cache->heads;
  p.G = q->heads / cache->heads;
  p.g_magic = p.G > 1 && static_cast<int64_t>(n) * p.G * p.G < (int64_t{1} << 32)
                  ? static_cast<uint32_t>((uint64_t{1} << 32) / p.G + 1)
                  : 0u;
  p.lens = lens;
  p.max_len = max_len;
  p.key_mask = key_mask;
  p.mask_stride = mask_stride;
  p.scale_log2 = scale * dllm::kLog2e;
  p.causal = causal != 0;
  p.B = B;
  p.n = n;
  return p;
}

// A matrix of words, one row a sequence.
dllm_status check_rows(const void* x, int64_t stride, int32_t B, int32_t max_len, const char* what) {
  if (!aligned(x, 4)) return fail(DLLM_ERR_INVALID_ARG, "%s must be 4-byte aligned", what);
  if (x && B > 1 && stride < max_len)
    return fail(DLLM_ERR_INVALID_ARG, "%s: stride %lld < max_len %d", what,
                static_cast<long long>(stride), max_len);
  return DLLM_OK;
}

dllm_status check_entries(int32_t B, int32_t max_len) {
  if (static_cast<int64_t>(B) * max_len > (int64_t{1} << 36))
    return fail(DLLM_ERR_UNSUPPORTED, "B * max_len exceeds 2^36");
  return DLLM_OK;
}

dllm_status check_evict(const dllm_kv4_cache* cache, int32_t B, int32_t max_len) {
  DLLM_TRY(check_cache(cache));
  DLLM_TRY(check_tokens(B, 1));
  if (max_len < 0 || max_len > static_cast<int64_t>(cache->table_stride) * cache->page_size)
    return fail(DLLM_ERR_INVALID_ARG, "max_len=%d outside [0, table_stride * page_size]", max_len);
  if (max_len > (1 << 30)) return fail(DLLM_ERR_UNSUPPORTED, "max_len=%d exceeds 2^30", max_len);
  return check_entries(B, max_len);
}

}  // namespace

namespace dllm {
void set_last_error(const char* msg, cudaError_t e) {
  if (e != cudaSuccess)
    snprintf(g_err, sizeof(g_err), "%s: %s", msg, cudaGetErrorString(e));
  else
    snprintf(g_err, sizeof(g_err), "%s", msg);
}
}  // namespace dllm

extern "C" {

const char* dllm_last_error(void) { return g_err; }

size_t dllm_workspace_bytes(const dllm_shape* shape) {
  if (check_shape(shape) != DLLM_OK) return 0;
  return dllm::stats_ws_bytes(shape->B, shape->L, shape->V);
}

dllm_status dllm_decode_stats(const void* logits, const dllm_shape* shape, const uint8_t* masked,
                              const dllm_stats* out, void* ws, dllm_stream_t stream) {
  CallRange range_("dllm_decode_stats");
  DLLM_TRY(check_shape(shape));
  if (!logits) return fail(DLLM_ERR_INVALID_ARG, "logits is null");
  DLLM_TRY(check_logits(logits, shape));
  DLLM_TRY(check_stats(out));
  DLLM_TRY(check_ws(ws));
  dllm::CommitArgs ca{};
  ca.mode = dllm::kStatsOnly;
  const dllm::StatsWs w = dllm::stats_ws_layout(ws, shape->B, shape->L, shape->V);
  cudaError_t e = dllm::launch_stats_commit(logits, *shape, masked, *out, nullptr, ca, w,
                                            sm_count(), reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_decode_stats");
  return ok();
}

dllm_status dllm_sample(const void* logits, const dllm_shape* shape, const uint8_t* masked,
                        const float* uniform, const dllm_sampling* how, const dllm_stats* out,
                        dllm_stream_t stream) {
  CallRange range_("dllm_sample");
  if (!logits) return fail(DLLM_ERR_INVALID_ARG, "logits is null");
  DLLM_TRY(check_shape(shape));
  DLLM_TRY(check_logits(logits, shape));
  DLLM_TRY(check_stats(out));
  if (!how || !uniform) return fail(DLLM_ERR_INVALID_ARG, "how and uniform must not be null");
  if (!aligned(uniform, 4)) return fail(DLLM_ERR_INVALID_ARG, "uniform must be 4-byte aligned");
  if (shape->V > (1 << 20)) return fail(DLLM_ERR_UNSUPPORTED, "V=%d exceeds 2^20", shape->V);
  const float t = how->temperature;
  if (t != 0.f && !(t >= 0x1p-10f && t <= 0x1p10f))
    return fail(DLLM_ERR_INVALID_ARG, "temperature %g is neither 0 nor in [2^-10, 2^10]", t);
  if (how->top_k < 0) return fail(DLLM_ERR_INVALID_ARG, "top_k=%d is negative", how->top_k);
  if (!(how->top_p > 0.f && how->top_p <= 1.f))
    return fail(DLLM_ERR_INVALID_ARG, "top_p %g is not in (0, 1]", how->top_p);
  if (!(how->min_p >= 0.f && how->min_p <= 1.f))
    return fail(DLLM_ERR_INVALID_ARG, "min_p %g is not in [0, 1]", how->min_p);
  cudaError_t e = dllm::launch_sample(logits, *shape, masked, uniform, *how, *out, sm_count(),
                                      reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_sample");
  return ok();
}

dllm_status dllm_commit_threshold(const void* logits, const dllm_shape* shape,
                                  const dllm_stats* stats, const dllm_block_state* state,
                                  float tau, int32_t eos_id, void* ws, dllm_stream_t stream) {
  CallRange range_("dllm_commit_threshold");
  return commit_common(logits, shape, stats, state, threshold_args(tau, eos_id), ws, stream,
                       "dllm_commit_threshold");
}

dllm_status dllm_commit_hierarchical(const void* logits, const dllm_shape* shape,
                                     const dllm_stats* stats, const dllm_block_state* state,
                                     float tau_low, int32_t min_width, int32_t eos_id, void* ws,
                                     dllm_stream_t stream) {
  CallRange range_("dllm_commit_hierarchical");
  if (min_width < 1) return fail(DLLM_ERR_INVALID_ARG, "min_width must be >= 1");
  dllm::CommitArgs ca{};
  ca.mode = dllm::kHierarchical;
  ca.tau_low = tau_low;
  ca.min_width = min_width;
  ca.eos_id = eos_id;
  return commit_common(logits, shape, stats, state, ca, ws, stream, "dllm_commit_hierarchical");
}

dllm_status dllm_commit_credit(const void* logits, const dllm_shape* shape,
                               const dllm_stats* stats, const dllm_block_state* state,
                               int32_t* cand_id, float* cand_credit, int32_t K, float decay,
                               float boost, float tau, int32_t eos_id, void* ws,
                               dllm_stream_t stream) {
  CallRange range_("dllm_commit_credit");
  if (!cand_id || !cand_credit)
    return fail(DLLM_ERR_INVALID_ARG, "cand_id and cand_credit must not be null");
  if (K < 1 || K > dllm::kMaxK)
    return fail(K < 1 ? DLLM_ERR_INVALID_ARG : DLLM_ERR_UNSUPPORTED, "K=%d outside [1, %d]", K,
                dllm::kMaxK);
  dllm::CommitArgs ca{};
  ca.mode = dllm::kCredit;
  ca.tau = tau;
  ca.eos_id = eos_id;
  ca.cand_id = cand_id;
  ca.cand_credit = cand_credit;
  ca.K = K;
  ca.decay = decay;
  ca.boost = boost;
  return commit_common(logits, shape, stats, state, ca, ws, stream, "dllm_commit_credit");
}

dllm_status dllm_commit_hierarchical_levels(const void* logits, const dllm_shape* shape,
                                            const dllm_stats* stats,
                                            const dllm_block_state* state, float tau_low,
                                            int32_t min_width, int32_t eos_id, void* ws,
                                            dllm_stream_t stream) {
  CallRange range_("dllm_commit_hierarchical_levels");
  if (min_width < 1) return fail(DLLM_ERR_INVALID_ARG, "min_width must be >= 1");
  dllm::CommitArgs ca{};
  ca.mode = dllm::kHierarchicalLevels;
  ca.tau_low = tau_low;
  ca.min_width = min_width;
  ca.eos_id = eos_id;
  return commit_common(logits, shape, stats, state, ca, ws, stream,
                       "dllm_commit_hierarchical_levels");
}

dllm_status dllm_commit_credit_tracked(const void* logits, const dllm_shape* shape,
                                       const dllm_stats* stats, const dllm_block_state* state,
                                       int32_t* cand_id, float* cand_credit, int32_t K,
                                       float decay, float boost, float tau, int32_t eos_id,
                                       void* ws, dllm_stream_t stream) {
  CallRange range_("dllm_commit_credit_tracked");
  if (!logits)
    return fail(DLLM_ERR_INVALID_ARG,
                "logits is null (the tracked-credit variant reads every tracked token's logit)");
  if (!cand_id || !cand_credit)
    return fail(DLLM_ERR_INVALID_ARG, "cand_id and cand_credit must not be null");
  if (K < 1 || K > dllm::kMaxK)
    return fail(K < 1 ? DLLM_ERR_INVALID_ARG : DLLM_ERR_UNSUPPORTED, "K=%d outside [1, %d]", K,
                dllm::kMaxK);
  dllm::CommitArgs ca{};
  ca.mode = dllm::kCreditTracked;
  ca.tau = tau;
  ca.eos_id = eos_id;
  ca.cand_id = cand_id;
  ca.cand_credit = cand_credit;
  ca.K = K;
  ca.decay = decay;
  ca.boost = boost;
  return commit_common(logits, shape, stats, state, ca, ws, stream, "dllm_commit_credit_tracked");
}

size_t dllm_embedding_t_elems(int32_t V, int32_t d) {
  if (V < 1 || d < 1) return 0;
  return static_cast<size_t>(d) * dllm::align_up(static_cast<size_t>(V), 64);
}

dllm_status dllm_prepare_embedding(const uint16_t* E, int32_t V, int32_t d, uint16_t* Et,
                                   dllm_stream_t stream) {
  CallRange range_("dllm_prepare_embedding");
  if (!E || !Et) return fail(DLLM_ERR_INVALID_ARG, "E and Et must not be null");
  if (V < 1 || d < 1) return fail(DLLM_ERR_INVALID_ARG, "V and d must be positive");
  if (d % 16 != 0) return fail(DLLM_ERR_UNSUPPORTED, "d=%d is not a multiple of 16", d);
  if (!aligned(Et, 16)) return fail(DLLM_ERR_INVALID_ARG, "Et must be 16-byte aligned");
  const int Vp = static_cast<int>(dllm::align_up(static_cast<size_t>(V), 64));
  cudaError_t e = dllm::launch_transpose_embedding(E, V, d, Et, Vp,
                                                   reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_prepare_embedding");
  return ok();
}

size_t dllm_smooth_workspace_bytes(const dllm_shape* shape, int32_t d) {
  if (check_shape(shape) != DLLM_OK || d < 16 || d % 16 != 0) return 0;
  return dllm::smooth_plan(shape->B, shape->L, shape->V, d, sm_count()).ws_bytes;
}

namespace {

dllm_status smooth_check(const dllm_shape* shape, int32_t d, void* ws, size_t ws_bytes,
                         dllm::SmoothPlan* pl) {
  DLLM_TRY(check_shape(shape));
  DLLM_TRY(check_ws(ws));
  if (d < 16 || d % 16 != 0 || d > 65536)
    return fail(DLLM_ERR_UNSUPPORTED, "d=%d must be a multiple of 16 in [16, 65536]", d);
  *pl = dllm::smooth_plan(shape->B, shape->L, shape->V, d, sm_count());
  if (ws_bytes < pl->ws_bytes)
    return fail(DLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed",
                ws_bytes, pl->ws_bytes);
  return DLLM_OK;
}

}  // namespace

dllm_status dllm_smooth_plan_info(const dllm_shape* shape, int32_t d, int32_t* info) {
  CallRange range_("dllm_smooth_plan_info");
  DLLM_TRY(check_shape(shape));
  if (!info) return fail(DLLM_ERR_INVALID_ARG, "info is null");
  if (d < 16 || d % 16 != 0 || d > 65536)
    return fail(DLLM_ERR_UNSUPPORTED, "d=%d must be a multiple of 16 in [16, 65536]", d);
  const dllm::SmoothPlan pl = dllm::smooth_plan(shape->B, shape->L, shape->V, d, sm_count());
  info[0] = pl.m_tiles;
  info[1] = pl.n_tiles;
  info[2] = pl.bn_max;
  info[3] = pl.partials;
  info[4] = pl.stages;
  info[5] = 3 + (pl.partials > 1 ? 1 : 0);  // rows, probabilities, GEMM (+ partial-sum reduction)
  return ok();
}

dllm_status dllm_smooth_probs(const void* logits, const dllm_shape* shape, const dllm_stats* stats,
                              const dllm_block_state* state, int32_t d, int32_t* row_ids,
                              int32_t* M, void* ws, size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_smooth_probs");
  dllm::SmoothPlan pl;
  DLLM_TRY(smooth_check(shape, d, ws, ws_bytes, &pl));
  if (!logits) return fail(DLLM_ERR_INVALID_ARG, "logits is null");
  DLLM_TRY(check_logits(logits, shape));
  DLLM_TRY(check_stats(stats));
  DLLM_TRY(check_state(state));
  if (!row_ids || !M) return fail(DLLM_ERR_INVALID_ARG, "row_ids and M must not be null");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint16_t* P = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + pl.off_p);
  cudaError_t e = dllm::launch_compact_rows(*state, shape->B, shape->L, row_ids, M, st);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_smooth_probs (rows)");
  e = dllm::launch_prob_rows(logits, *shape, stats->lse, row_ids, M, P, pl.m_tiles * 128,
                             sm_count(), st);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_smooth_probs (probabilities)");
  return ok();
}

dllm_status dllm_smooth_gemm(const dllm_shape* shape, const uint16_t* Et, int32_t d, float* out,
                             const int32_t* M, void* ws, size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_smooth_gemm");
  dllm::SmoothPlan pl;
  DLLM_TRY(smooth_check(shape, d, ws, ws_bytes, &pl));
  if (!Et || !out || !M) return fail(DLLM_ERR_INVALID_ARG, "Et, out and M must not be null");
  if (!aligned(Et, 16) || !aligned(out, 16))
    return fail(DLLM_ERR_INVALID_ARG, "Et and out must be 16-byte aligned");
  const uint16_t* P =
      reinterpret_cast<const uint16_t*>(static_cast<const char*>(ws) + pl.off_p);
  const char* why = "launch failed";
  const int ldt = static_cast<int>(dllm::align_up(static_cast<size_t>(shape->V), 8));
  cudaError_t e = dllm::launch_smooth_gemm(pl, P, Et, ldt, out, M, nullptr, false, ws,
                                           reinterpret_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess)
    return fail(DLLM_ERR_CUDA, "dllm_smooth_gemm: %s: %s", why, cudaGetErrorString(e));
  return ok();
}

dllm_status dllm_smooth_embed(const void* logits, const dllm_shape* shape, const dllm_stats* stats,
                              const dllm_block_state* state, const uint16_t* Et, int32_t d,
                              float* out, int32_t* row_ids, int32_t* M, void* ws,
                              size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_smooth_embed");
  if (!Et || !out) return fail(DLLM_ERR_INVALID_ARG, "Et and out must not be null");
  if (!aligned(Et, 16) || !aligned(out, 16))
    return fail(DLLM_ERR_INVALID_ARG, "Et and out must be 16-byte aligned");
  DLLM_TRY(dllm_smooth_probs(logits, shape, stats, state, d, row_ids, M, ws, ws_bytes, stream));
  return dllm_smooth_gemm(shape, Et, d, out, M, ws, ws_bytes, stream);
}

dllm_status dllm_commit_threshold_smooth(const void* logits, const dllm_shape* shape,
                                        const dllm_stats* stats, const dllm_block_state* state,
                                        float tau, int32_t eos_id, const uint16_t* Et, int32_t d,
                                        float* out, int32_t* row_ids, int32_t* M, void* ws,
                                        size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_commit_threshold_smooth");
  dllm::SmoothPlan pl;
  DLLM_TRY(smooth_check(shape, d, ws, ws_bytes, &pl));
  if (!logits) return fail(DLLM_ERR_INVALID_ARG, "logits is null");
  DLLM_TRY(check_logits(logits, shape));
  DLLM_TRY(check_stats(stats));
  DLLM_TRY(check_state(state));
  if (!Et || !out || !row_ids || !M)
    return fail(DLLM_ERR_INVALID_ARG, "Et, out, row_ids and M must not be null");
  if (!aligned(Et, 16) || !aligned(out, 16))
    return fail(DLLM_ERR_INVALID_ARG, "Et and out must be 16-byte aligned");
  int C = 0, per = 0;
  if (!rows_vector_aligned(logits, shape) ||
      !dllm::stats_probs_split(shape->V, shape->dtype, &C, &per)) {
    // rows the single-read kernels cannot copy whole (not 16-byte aligned, V not a multiple of
    // 8, or longer than 8 x 192 KB): the same results from the separate calls, which read such
    // rows element by element (the logits are read twice)
    DLLM_TRY(commit_common(logits, shape, stats, state, threshold_args(tau, eos_id),
                           static_cast<char*>(ws) + pl.off_stats_ws, stream,
                           "dllm_commit_threshold_smooth"));
    return dllm_smooth_embed(logits, shape, stats, state, Et, d, out, row_ids, M, ws, ws_bytes,
                             stream);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  uint16_t* P = reinterpret_cast<uint16_t*>(w + pl.off_p);
  int32_t* rows = reinterpret_cast<int32_t*>(w + pl.off_rows);
  int32_t* count = reinterpret_cast<int32_t*>(w + pl.off_count);
  int32_t* inv = reinterpret_cast<int32_t*>(w + pl.off_inv);
  int32_t* map = reinterpret_cast<int32_t*>(w + pl.off_map);
  const int R_pad = pl.m_tiles * 128;
  cudaError_t e = dllm::launch_read_rows(*state, shape->B, shape->L, rows, count, *stats, st);
  if (e == cudaSuccess)
    e = dllm::launch_stats_probs(logits, *shape, rows, count, *stats, P, R_pad,
                                 static_cast<int32_t*>(ws), st);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_commit_threshold_smooth (statistics)");
  dllm::CommitArgs ca{};
  ca.mode = dllm::kThreshold;
  ca.tau = tau;
  ca.eos_id = eos_id;
  e = dllm::launch_commit_only(*shape, *stats, *state, ca, st);
  if (e == cudaSuccess)
    e = dllm::launch_kept_rows_map(*state, shape->B, shape->L, row_ids, M, rows, count, inv, map,
                                   st);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_commit_threshold_smooth (commit)");
  const char* why = "launch failed";
  const int ldt = static_cast<int>(dllm::align_up(static_cast<size_t>(shape->V), 8));
  // P (statistics kernel) and count (row list) predate the kept-row map, the only input the
  // kernel just before the GEMM writes: the GEMM's mainloop overlaps it
  e = dllm::launch_smooth_gemm(pl, P, Et, ldt, out, count, map, true, ws, st, &why);
  if (e != cudaSuccess)
    return fail(DLLM_ERR_CUDA, "dllm_commit_threshold_smooth: %s: %s", why,
                cudaGetErrorString(e));
  return ok();
}

dllm_status dllm_block_state_reset(const dllm_block_state* state, int32_t B, int32_t L,
                                   int32_t* cand_id, float* cand_credit, int32_t K,
                                   dllm_stream_t stream) {
  CallRange range_("dllm_block_state_reset");
  DLLM_TRY(check_state(state));
  if (B < 1 || L < 1) return fail(DLLM_ERR_INVALID_ARG, "need B, L >= 1 (B=%d L=%d)", B, L);
  if (L > dllm::kMaxL) return fail(DLLM_ERR_UNSUPPORTED, "L=%d exceeds %d", L, dllm::kMaxL);
  if (static_cast<int64_t>(B) * L > (int64_t{1} << 20))
    return fail(DLLM_ERR_UNSUPPORTED, "B*L=%lld exceeds 2^20",
                static_cast<long long>(B) * L);
  const bool credit = cand_id != nullptr || cand_credit != nullptr;
  if (credit && (K < 1 || K > dllm::kMaxK))
    return fail(DLLM_ERR_INVALID_ARG, "K=%d must be in [1, %d] with credit slots", K,
                dllm::kMaxK);
  const int64_t n = static_cast<int64_t>(B) * L;
  cudaError_t e = dllm::launch_block_state_reset(*state, n, B, cand_id, cand_credit,
                                                 credit ? n * K : 0,
                                                 reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_block_state_reset");
  return ok();
}

dllm_status dllm_capture_condition(dllm_stream_t stream, uint32_t default_value,
                                   uint64_t* handle_out) {
  CallRange range_("dllm_capture_condition");
  if (!handle_out) return fail(DLLM_ERR_INVALID_ARG, "handle_out is null");
  cudaGraph_t graph = nullptr;
  DLLM_TRY(capturing_graph(stream, &graph, nullptr, nullptr, "dllm_capture_condition"));
  cudaGraphConditionalHandle h = 0;
  cudaError_t e = cudaGraphConditionalHandleCreate(&h, graph, default_value ? 1u : 0u,
                                                   cudaGraphCondAssignDefault);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_capture_condition");
  *handle_out = static_cast<uint64_t>(h);
  return ok();
}

dllm_status dllm_capture_if_begin(dllm_stream_t stream, dllm_stream_t body_stream,
                                  uint64_t handle) {
  CallRange range_("dllm_capture_if_begin");
  if (stream == body_stream)
    return fail(DLLM_ERR_INVALID_ARG, "the conditional body needs a stream of its own");
  cudaGraph_t graph = nullptr;
  const cudaGraphNode_t* deps = nullptr;
  size_t n_deps = 0;
  DLLM_TRY(capturing_graph(stream, &graph, &deps, &n_deps, "dllm_capture_if_begin"));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaStream_t bs = reinterpret_cast<cudaStream_t>(body_stream);
  cudaStreamCaptureStatus bcs = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(bs, &bcs);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_capture_if_begin (body stream)");
  if (bcs != cudaStreamCaptureStatusNone)
    return fail(DLLM_ERR_INVALID_ARG, "body_stream is already capturing");
  cudaGraphNodeParams np = {};
  np.type = cudaGraphNodeTypeConditional;
  np.conditional.handle = static_cast<cudaGraphConditionalHandle>(handle);
  np.conditional.type = cudaGraphCondTypeIf;
  np.conditional.size = 1;
  cudaGraphNode_t node = nullptr;
  e = cudaGraphAddNode(&node, graph, deps, nullptr, n_deps, &np);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_capture_if_begin (conditional node)");
  // later work on `stream` follows the node; the body is captured on body_stream
  e = cudaStreamUpdateCaptureDependencies(s, &node, nullptr, 1, cudaStreamSetCaptureDependencies);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_capture_if_begin (dependencies)");
  e = cudaStreamBeginCaptureToGraph(bs, np.conditional.phGraph_out[0], nullptr, nullptr, 0,
                                    cudaStreamCaptureModeRelaxed);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_capture_if_begin (body capture)");
  return ok();
}

dllm_status dllm_capture_if_end(dllm_stream_t body_stream) {
  CallRange range_("dllm_capture_if_end");
  cudaGraph_t body = nullptr;  // owned by the conditional node
  cudaError_t e = cudaStreamEndCapture(reinterpret_cast<cudaStream_t>(body_stream), &body);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_capture_if_end");
  return ok();
}

dllm_status dllm_loop_continue(const dllm_block_state* state, int32_t B, int32_t L,
                               uint64_t handle, dllm_stream_t stream) {
  CallRange range_("dllm_loop_continue");
  if (!state || !state->masked || !state->eos_hit)
    return fail(DLLM_ERR_INVALID_ARG, "state.masked and state.eos_hit must not be null");
  if (B < 1 || L < 1) return fail(DLLM_ERR_INVALID_ARG, "need B, L >= 1 (B=%d L=%d)", B, L);
  if (L > dllm::kMaxL) return fail(DLLM_ERR_UNSUPPORTED, "L=%d exceeds %d", L, dllm::kMaxL);
  if (static_cast<int64_t>(B) * L > (int64_t{1} << 20))
    return fail(DLLM_ERR_UNSUPPORTED, "B*L=%lld exceeds 2^20", static_cast<long long>(B) * L);
  cudaGraph_t graph = nullptr;  // the handle exists only inside its graph
  DLLM_TRY(capturing_graph(stream, &graph, nullptr, nullptr, "dllm_loop_continue"));
  cudaError_t e = dllm::launch_loop_continue(*state, B, L,
                                             static_cast<cudaGraphConditionalHandle>(handle),
                                             reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_loop_continue");
  return ok();
}

dllm_status dllm_kv_refresh_mask(const dllm_block_state* state, int32_t B, int32_t L,
                                 int32_t prefix_len, int32_t window, uint8_t* refresh,
                                 int32_t* idx, int32_t* count, dllm_stream_t stream) {
  CallRange range_("dllm_kv_refresh_mask");
  if (!state || !state->committed_now)
    return fail(DLLM_ERR_INVALID_ARG, "state.committed_now is null");
  if (!refresh || !idx || !count)
    return fail(DLLM_ERR_INVALID_ARG, "refresh, idx and count must not be null");
  if (B < 1 || L < 1 || prefix_len < 0 || window < 0)
    return fail(DLLM_ERR_INVALID_ARG, "need B, L >= 1 and prefix_len, window >= 0");
  if (static_cast<int64_t>(prefix_len) + L > 65536)
    return fail(DLLM_ERR_UNSUPPORTED, "prefix_len + L exceeds 65536");
  if (L > dllm::kMaxL) return fail(DLLM_ERR_UNSUPPORTED, "L=%d exceeds %d", L, dllm::kMaxL);
  cudaError_t e = dllm::launch_kv_refresh(*state, B, L, prefix_len, window, refresh, idx, count,
                                          reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_kv_refresh_mask");
  return ok();
}

dllm_status dllm_selftest_wait_timeout(void* ws, uint32_t limit_us, dllm_stream_t stream) {
  CallRange range_("dllm_selftest_wait_timeout");
  DLLM_TRY(check_ws(ws));
  if (limit_us < 1 || limit_us > 2000000)
    return fail(DLLM_ERR_INVALID_ARG, "limit_us must be in [1, 2000000]");
  cudaError_t e = dllm::launch_wait_timeout_selftest(static_cast<int32_t*>(ws),
                                                     static_cast<uint64_t>(limit_us) * 1000,
                                                     reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_selftest_wait_timeout");
  return ok();
}

dllm_status dllm_merge_shard_stats(const dllm_shard_stats* shards, int32_t n, int64_t rows,
                                   const dllm_stats* out, dllm_stream_t stream) {
  CallRange range_("dllm_merge_shard_stats");
  if (!shards) return fail(DLLM_ERR_INVALID_ARG, "shards is null");
  if (n < 1 || n > DLLM_MAX_SHARDS)
    return fail(DLLM_ERR_INVALID_ARG, "n=%d must be in [1, %d]", n, DLLM_MAX_SHARDS);
  if (rows < 0 || rows > (int64_t{1} << 31))
    return fail(DLLM_ERR_INVALID_ARG, "rows=%lld out of range", static_cast<long long>(rows));
  DLLM_TRY(check_stats(out));
  for (int k = 0; k < n; ++k) {
    DLLM_TRY(check_stats(&shards[k].stats));
    if (shards[k].vocab_offset < 0 || shards[k].vocab_offset >= (int64_t{1} << 31))
      return fail(DLLM_ERR_INVALID_ARG, "shard %d: vocab_offset out of range", k);
    const dllm_stats& a = shards[k].stats;
    if (a.row_max == out->row_max || a.lse == out->lse || a.conf == out->conf ||
        a.argmax == out->argmax)
      return fail(DLLM_ERR_INVALID_ARG, "shard %d aliases the output", k);
  }
  cudaError_t e = dllm::launch_merge_shard_stats(shards, n, rows, *out,
                                                 reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_merge_shard_stats");
  return ok();
}

dllm_status dllm_rope_phases(const dllm_rope* rope, int64_t* phases, dllm_stream_t stream) {
  CallRange range_("dllm_rope_phases");
  if (!rope || !phases) return fail(DLLM_ERR_INVALID_ARG, "rope and phases must not be null");
  if (!aligned(phases, 8)) return fail(DLLM_ERR_INVALID_ARG, "phases must be 8-byte aligned");
  if (rope->rotary_dim < 2 || rope->rotary_dim % 2 != 0)
    return fail(DLLM_ERR_INVALID_ARG, "rotary_dim=%d must be even and positive", rope->rotary_dim);
  if (rope->rotary_dim > 1024)
    return fail(DLLM_ERR_UNSUPPORTED, "rotary_dim=%d exceeds 1024", rope->rotary_dim);
  if (rope->scaling != DLLM_ROPE_LINEAR && rope->scaling != DLLM_ROPE_BANDS)
    return fail(DLLM_ERR_UNSUPPORTED, "scaling %d is not LINEAR (0) or BANDS (1)", rope->scaling);
  if (!(rope->base > 1.0) || !std::isfinite(rope->base) || !(rope->factor >= 1.0) ||
      !std::isfinite(rope->factor))
    return fail(DLLM_ERR_INVALID_ARG, "need a finite base > 1 and factor >= 1");
  if (rope->scaling == DLLM_ROPE_BANDS &&
      (!(rope->original_len > 0.0) || !std::isfinite(rope->original_len) ||
       !(rope->slow_turns >= 0.0) || !(rope->fast_turns > rope->slow_turns) ||
       !std::isfinite(rope->fast_turns)))
    return fail(DLLM_ERR_INVALID_ARG,
                "need original_len > 0 and 0 <= slow_turns < fast_turns, all finite");
  cudaError_t e = dllm::launch_rope_phases(*rope, phases, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_rope_phases");
  return ok();
}

dllm_status dllm_qk_norm_rope(const dllm_heads* q, const dllm_heads* q_out, const dllm_heads* k,
                              const dllm_heads* k_out, int32_t B, int32_t n, int32_t head_dim,
                              const int32_t* pos, int64_t pos_stride, const int64_t* phases,
                              int32_t rotary_dim, int32_t interleaved, float magnitude,
                              int32_t norm, const void* q_weight, const void* k_weight, float eps,
                              dllm_stream_t stream) {
  CallRange range_("dllm_qk_norm_rope");
  if (!q != !q_out || !k != !k_out || (!q && !k))
    return fail(DLLM_ERR_INVALID_ARG, "need q with q_out, or k with k_out, or both pairs");
  int dtype = -1;
  const dllm_heads* in[2] = {q, k};
  const dllm_heads* out[2] = {q_out, k_out};
  for (int j = 0; j < 2; ++j) {
    if (!in[j]) continue;
    DLLM_TRY(check_heads(in[j], j ? "k" : "q"));
    DLLM_TRY(check_heads(out[j], j ? "k_out" : "q_out"));
    if (in[j]->heads != out[j]->heads)
      return fail(DLLM_ERR_INVALID_ARG, "%s and its output differ in heads", j ? "k" : "q");
    if (dtype < 0) dtype = in[j]->dtype;
    if (in[j]->dtype != dtype || out[j]->dtype != dtype)
      return fail(DLLM_ERR_INVALID_ARG, "the tensors differ in dtype");
  }
  DLLM_TRY(check_tokens(B, n));
  // a warp each in the largest grid of four-warp blocks
  const int64_t rows = static_cast<int64_t>(B) * n * ((q ? q->heads : 0) + (k ? k->heads : 0));
  if (rows > (int64_t{1} << 33) - 4)
    return fail(DLLM_ERR_UNSUPPORTED, "B*n tokens of all heads: %lld exceeds 2^33 - 4",
                static_cast<long long>(rows));
  if (head_dim < 1 || head_dim > 1024)
    return fail(head_dim < 1 ? DLLM_ERR_INVALID_ARG : DLLM_ERR_UNSUPPORTED,
                "head_dim=%d outside [1, 1024]", head_dim);
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim)
    return fail(DLLM_ERR_INVALID_ARG, "rotary_dim=%d must be even and in [0, head_dim=%d]",
                rotary_dim, head_dim);
  if (rotary_dim > 0 && (!pos || !phases))
    return fail(DLLM_ERR_INVALID_ARG, "a rotation needs pos and phases");
  if (rotary_dim == 0 && !norm)
    return fail(DLLM_ERR_INVALID_ARG, "neither a norm nor a rotation is asked for");
  if (norm && !(eps >= 0.f)) return fail(DLLM_ERR_INVALID_ARG, "eps must be >= 0");
  if (!norm && (q_weight || k_weight))
    return fail(DLLM_ERR_INVALID_ARG, "weights without a norm");
  const size_t es = dtype == DLLM_BF16 ? 2 : 4;
  if (!aligned(q_weight, es) || !aligned(k_weight, es) || !aligned(pos, 4) || !aligned(phases, 8))
    return fail(DLLM_ERR_INVALID_ARG, "weights, pos and phases must be aligned to their elements");
  cudaError_t e = dllm::launch_norm_rope(
      q, q_out, k, k_out, B, n, head_dim, pos, pos_stride, phases, rotary_dim, interleaved != 0,
      magnitude, norm != 0, q_weight, k_weight, eps, sm_count(),
      reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_qk_norm_rope");
  return ok();
}

dllm_status dllm_kv4_write(const dllm_kv4_cache* cache, const dllm_heads* k, const dllm_heads* v,
                           int32_t B, int32_t n, const int32_t* pos, int64_t pos_stride,
                           dllm_stream_t stream) {
  CallRange range_("dllm_kv4_write");
  DLLM_TRY(check_cache_rows(cache, k, v, B, n));
  if (!pos || !aligned(pos, 4))
    return fail(DLLM_ERR_INVALID_ARG, "pos must not be null and 4-byte aligned");
  cudaError_t e = dllm::launch_kv4_write(*cache, *k, *v, B, n, pos, pos_stride, sm_count(),
                                         reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_kv4_write");
  return ok();
}

dllm_status dllm_kv4_read(const dllm_kv4_cache* cache, const dllm_heads* k, const dllm_heads* v,
                          int32_t B, int32_t n, const int32_t* pos, int64_t pos_stride,
                          dllm_stream_t stream) {
  CallRange range_("dllm_kv4_read");
  DLLM_TRY(check_cache_rows(cache, k, v, B, n));
  if (!aligned(pos, 4)) return fail(DLLM_ERR_INVALID_ARG, "pos must be 4-byte aligned");
  cudaError_t e = dllm::launch_kv4_read(*cache, *k, *v, B, n, pos, pos_stride, sm_count(),
                                        reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_kv4_read");
  return ok();
}

size_t dllm_attention_kv4_workspace_bytes(const dllm_kv4_cache* cache, int32_t B, int32_t n,
                                          int32_t q_heads, int32_t max_len) {
  if (check_attention(cache, B, n, q_heads, max_len) != DLLM_OK) return 0;
  return dllm::attention_ws_bytes(B, n, q_heads / cache->heads, cache->heads, cache->head_dim,
                                  max_len, sm_count());
}

dllm_status dllm_attention_kv4(const dllm_heads* q, const dllm_kv4_cache* cache,
                               const int32_t* lens, int32_t max_len, const uint8_t* key_mask,
                               int64_t mask_stride, float scale, int32_t causal,
                               const dllm_heads* out, float* lse, int32_t B, int32_t n, void* ws,
                               size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_attention_kv4");
  DLLM_TRY(check_heads(q, "q"));
  DLLM_TRY(check_heads(out, "out"));
  DLLM_TRY(check_attention(cache, B, n, q->heads, max_len));
  DLLM_TRY(check_ws(ws));
  if (q->dtype != DLLM_BF16 || out->dtype != DLLM_BF16)
    return fail(DLLM_ERR_UNSUPPORTED, "q and out must be bf16");
  if (q->heads != out->heads)
    return fail(DLLM_ERR_INVALID_ARG, "q has %d heads, out %d", q->heads, out->heads);
  if (!std::isfinite(scale)) return fail(DLLM_ERR_INVALID_ARG, "scale is not finite");
  if (key_mask && B > 1 && mask_stride != 0 && mask_stride < max_len)
    return fail(DLLM_ERR_INVALID_ARG, "mask_stride %lld < max_len %d",
                static_cast<long long>(mask_stride), max_len);
  if (!aligned(lens, 4) || !aligned(lse, 4))
    return fail(DLLM_ERR_INVALID_ARG, "lens and lse must be 4-byte aligned");
  const size_t need = dllm::attention_ws_bytes(B, n, q->heads / cache->heads, cache->heads,
                                               cache->head_dim, max_len, sm_count());
  if (ws_bytes < need)
    return fail(DLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed",
                ws_bytes, need);
  dllm::AttnParams p = attention_params(q, cache, lens, max_len, key_mask, mask_stride, scale, causal, B, n);
  p.out = static_cast<uint16_t*>(out->data);
  p.ob = out->batch_stride, p.ot = out->token_stride, p.oh = out->head_stride;
  p.lse = lse;
  cudaError_t e = dllm::launch_attention(p, cache->head_dim, ws, sm_count(),
                                         reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_attention_kv4");
  return ok();
}

size_t dllm_attention_kv4_weights_workspace_bytes(const dllm_kv4_cache* cache, int32_t B, int32_t n,
                                                  int32_t q_heads, int32_t max_len) {
  if (check_attention(cache, B, n, q_heads, max_len) != DLLM_OK || check_entries(B, max_len) != DLLM_OK)
    return 0;
  return dllm::attention_weights_ws_bytes(B, n, q_heads / cache->heads, cache->heads, cache->head_dim,
                                          max_len);
}

dllm_status dllm_attention_kv4_weights(const dllm_heads* q, const dllm_kv4_cache* cache,
                                       const int32_t* lens, int32_t max_len,
                                       const uint8_t* key_mask, int64_t mask_stride, float scale,
                                       int32_t causal, const float* lse, const float* prior,
                                       int64_t prior_stride, float keep, float* weights,
                                       int64_t weights_stride, int32_t B, int32_t n, void* ws,
                                       size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_attention_kv4_weights");
  DLLM_TRY(check_heads(q, "q"));
  DLLM_TRY(check_attention(cache, B, n, q->heads, max_len));
  DLLM_TRY(check_entries(B, max_len));
  DLLM_TRY(check_ws(ws));
  if (q->dtype != DLLM_BF16) return fail(DLLM_ERR_UNSUPPORTED, "q must be bf16");
  if (!lse || !weights) return fail(DLLM_ERR_INVALID_ARG, "lse and weights must not be null");
  if (!std::isfinite(scale)) return fail(DLLM_ERR_INVALID_ARG, "scale is not finite");
  if (prior && !std::isfinite(keep)) return fail(DLLM_ERR_INVALID_ARG, "keep is not finite");
  if (key_mask && B > 1 && mask_stride != 0 && mask_stride < max_len)
    return fail(DLLM_ERR_INVALID_ARG, "mask_stride %lld < max_len %d",
                static_cast<long long>(mask_stride), max_len);
  if (!aligned(lens, 4) || !aligned(lse, 4))
    return fail(DLLM_ERR_INVALID_ARG, "lens and lse must be 4-byte aligned");
  DLLM_TRY(check_rows(weights, weights_stride, B, max_len, "weights"));
  DLLM_TRY(check_rows(prior, prior_stride, B, max_len, "prior"));
  if (prior == weights && prior_stride != weights_stride && B > 1)
    return fail(DLLM_ERR_INVALID_ARG, "prior and weights are one memory with two strides");
  const size_t need = dllm::attention_weights_ws_bytes(B, n, q->heads / cache->heads, cache->heads,
                                                       cache->head_dim, max_len);
  if (ws_bytes < need)
    return fail(DLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes,
                need);
  const dllm::AttnParams p =
      attention_params(q, cache, lens, max_len, key_mask, mask_stride, scale, causal, B, n);
  dllm::AttnWeights x{};
  x.lse = lse;
  x.prior = prior;
  x.prior_stride = prior_stride;
  x.out = weights;
  x.out_stride = weights_stride;
  x.keep = keep;
  x.scale = scale;
  cudaError_t e = dllm::launch_attention_weights(p, x, cache->head_dim, ws, sm_count(),
                                                 reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_attention_kv4_weights");
  return ok();
}

size_t dllm_kv4_evict_workspace_bytes(const dllm_kv4_cache* cache, int32_t B, int32_t max_len) {
  return check_evict(cache, B, max_len) == DLLM_OK ? dllm::kv4_evict_ws_bytes(B, max_len) : 0;
}

dllm_status dllm_kv4_evict(const dllm_kv4_cache* cache, const float* weights, int64_t weights_stride,
                           const int32_t* lens, int32_t max_len, int32_t budget, int32_t first,
                           int32_t last, int32_t* slots, int64_t slots_stride, int32_t* lens_out,
                           float* weights_out, int64_t weights_out_stride, int32_t B, void* ws,
                           size_t ws_bytes, dllm_stream_t stream) {
  CallRange range_("dllm_kv4_evict");
  DLLM_TRY(check_evict(cache, B, max_len));
  DLLM_TRY(check_ws(ws));
  if (!weights || !slots || !lens_out)
    return fail(DLLM_ERR_INVALID_ARG, "weights, slots and lens_out must not be null");
  if (budget < 0 || first < 0 || last < 0 || static_cast<int64_t>(first) + last > budget)
    return fail(DLLM_ERR_INVALID_ARG,
                "need budget, first, last >= 0 and first + last <= budget (%d, %d, %d)", budget, first,
                last);
  if (!aligned(lens, 4) || !aligned(lens_out, 4))
    return fail(DLLM_ERR_INVALID_ARG, "lens and lens_out must be 4-byte aligned");
  DLLM_TRY(check_rows(weights, weights_stride, B, max_len, "weights"));
  DLLM_TRY(check_rows(slots, slots_stride, B, max_len, "slots"));
  DLLM_TRY(check_rows(weights_out, weights_out_stride, B, max_len, "weights_out"));
  if (weights_out == weights && weights_out_stride != weights_stride && B > 1)
    return fail(DLLM_ERR_INVALID_ARG, "weights and weights_out are one memory with two strides");
  const size_t need = dllm::kv4_evict_ws_bytes(B, max_len);
  if (ws_bytes < need)
    return fail(DLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes,
                need);
  cudaError_t e = dllm::launch_kv4_evict(*cache, weights, weights_stride, lens, max_len, budget, first,
                                         last, slots, slots_stride, lens_out, weights_out,
                                         weights_out_stride, B, ws, sm_count(),
                                         reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dllm_kv4_evict");
  return ok();
}

dllm_status dllm_get_status(void* ws, dllm_stream_t stream, int32_t* out_host) {
  CallRange range_("dllm_get_status");
  DLLM_TRY(check_ws(ws));
  if (!out_host) return fail(DLLM_ERR_INVALID_ARG, "out_host is null");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, ws, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "dllm_get_status");
  *out_host = v;
  if (v != DLLM_OK) {
    e = cudaMemsetAsync(ws, 0, sizeof(int32_t), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "dllm_get_status (reset)");
  }
  return ok();
}

}  // extern "C"
