/*
 * dllm.h — C ABI of the parallel-decode step of a diffusion language model, for NVIDIA GB300
 * (sm_103a).
 *
 * One decode iteration of a masked-diffusion LM ends with the model's logits for a block of L
 * positions in each of B sequences.  The step turns them into decisions: which still-masked
 * positions to fix ("commit") now and with which token, what to feed back for the positions
 * left open, and which KV-cache entries must be recomputed.  Sources, cited by page and
 * section:
 *   [dInfer explainer]  the 91haoming.cn summary of the dInfer paper (arXiv 2510.08666): its
 *                       decoding-strategy component (threshold, hierarchical and credit
 *                       decoding), diffusion-iteration manager (iteration smoothing), KV-cache
 *                       manager (neighbourhood refresh) and engineering notes (early stop).
 *   [dInfer news]       the aibase.com article: the four modules (model access, KV-cache
 *                       manager, diffusion-iteration manager, decoding strategies).
 * The pages give no formulas; the exact definitions these functions compute are restated at
 * each declaration.
 *
 * Conventions shared by every function:
 *  - Every pointer argument is DEVICE memory owned by the caller, except the `const dllm_*`
 *    descriptor structs themselves, `out_host` of dllm_get_status and `handle_out` of
 *    dllm_capture_condition, which are host memory read (or written) before the function
 *    returns.  The library never allocates or frees
 *    device memory and never synchronises the stream, except dllm_get_status.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) and runs
 *    asynchronously.  The functions hold no host state between calls, so a sequence of calls
 *    can be captured into a CUDA graph.
 *  - Return value: DLLM_OK when the work was enqueued.  DLLM_ERR_INVALID_ARG (a null pointer,
 *    a non-positive size, a misaligned pointer, a stride shorter than a row) and
 *    DLLM_ERR_UNSUPPORTED (a size beyond a documented limit) are returned before anything is
 *    launched.  DLLM_ERR_CUDA means a launch failed.  dllm_last_error() then describes the
 *    failure (thread-local, valid until the next call on the same thread).
 *  - Faults found while the kernels run (a wait that timed out inside the smoothing GEMM) are
 *    recorded in the status word at the start of the workspace; dllm_get_status reads it.
 *  - Workspace: `ws` points to at least dllm_workspace_bytes(shape) bytes (or
 *    dllm_smooth_workspace_bytes for dllm_smooth_embed), 256-byte aligned, zero-filled ONCE
 *    before its first use (its first 4 bytes are the status word).  The same workspace serves
 *    any number of later calls on one stream.  Calls that run at the same time must use
 *    different workspaces.
 *
 * Data layout (row r = b*L + i is position i of sequence b):
 *  - logits: B*L rows of V elements, row r starting at element r*row_stride; row_stride >= V.
 *    fp32 or bf16 (dllm_shape.dtype).  The pointer is aligned to the element size.  Rows that
 *    all start on 16-byte boundaries (pointer and row_stride * element size multiples of 16)
 *    are read with 16-byte vector loads; any other layout (and, for the smoothing calls, V not
 *    a multiple of 8) is read element by element by the same kernels (slower, same results).
 *  - block state (dllm_block_state), all [B, L] or [B] row-major:
 *      masked[B*L]        uint8, 1 = position still undecided;
 *      tokens[B*L]        int32, committed token id, -1 while masked;
 *      committed_now[B*L] uint8, written by every commit call: 1 = committed in this call;
 *      n_commit[B]        int32, written by every commit call: number committed in this call;
 *      eos_hit[B]         int32, set to 1 when a committed token equals eos_id; a sequence
 *                         with eos_hit set, or with nothing masked, is stopped: later calls do
 *                         not read its logits, commit nothing and leave its state untouched.
 *  - statistics (dllm_stats), [B*L] each: row_max (fp32), lse (fp32, natural log-sum-exp),
 *    conf (fp32, top-1 probability) and argmax (int32, lowest index of the maximum).  Rows not
 *    computed hold -inf, -inf, 0 and -1.
 */
#ifndef DLLM_H_
#define DLLM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* dllm_stream_t; /* same type as cudaStream_t */

typedef enum {
  DLLM_OK = 0,
  DLLM_ERR_INVALID_ARG = 1,
  DLLM_ERR_UNSUPPORTED = 2,
  DLLM_ERR_CUDA = 3,
  DLLM_ERR_TIMEOUT = 4
} dllm_status;

typedef enum { DLLM_F32 = 0, DLLM_BF16 = 1 } dllm_dtype;

/* Shape of one block of logits.  Limits: B >= 1, 1 <= L <= 1024, 2 <= V < 2^31,
 * B*L <= 2^20, row_stride >= V. */
typedef struct {
  int32_t B;
  int32_t L;
  int32_t V;
  int32_t dtype;      /* dllm_dtype */
  int64_t row_stride; /* elements between the starts of consecutive rows */
} dllm_shape;

typedef struct {
  uint8_t* masked;
  int32_t* tokens;
  uint8_t* committed_now;
  int32_t* n_commit;
  int32_t* eos_hit;
} dllm_block_state;

typedef struct {
  float* row_max;
  float* lse;
  float* conf;
  int32_t* argmax;
} dllm_stats;

/* Description of the last error on this thread ("" if none). */
const char* dllm_last_error(void);

/*
 * Start a new block (dInfer explainer, diffusion-iteration manager: a block starts with every
 * position masked and is decoded over iterations until filled or stopped): one kernel sets
 *   masked[B*L] = 1, tokens[B*L] = -1, committed_now[B*L] = 0, n_commit[B] = 0, eos_hit[B] = 0
 * and, when cand_id / cand_credit are not NULL (the credit-decoding state, [B*L, K] each),
 * cand_id = -1 (empty slot) and cand_credit = 0.  1 <= K <= 16 when either is given.
 * B >= 1, 1 <= L <= 1024, B*L <= 2^20.  Same stream rules as every call: it is ordered after
 * the calls before it on `stream`, so a decode loop with its reset can be captured whole.
 */
dllm_status dllm_block_state_reset(const dllm_block_state* state, int32_t B, int32_t L,
                                   int32_t* cand_id, float* cand_credit, int32_t K,
                                   dllm_stream_t stream);

/* Bytes of workspace the stats and commit calls need for `shape` (0 if shape is invalid). */
size_t dllm_workspace_bytes(const dllm_shape* shape);

/*
 * Softmax statistics of every row (dInfer explainer, decoding strategies: each strategy ranks
 * the undecided positions by the model's confidence in its top token).  For a computed row z:
 *   row_max = max_v z_v;  s = sum_v exp(z_v - row_max);  lse = row_max + ln s;
 *   conf = 1/s (the top-1 probability);  argmax = lowest v with z_v = row_max.
 * masked: [B*L] uint8 or NULL.  With a mask, only rows with masked[r] = 1 are read and
 * computed; with NULL every row is.  Each logit crosses HBM once.
 */
dllm_status dllm_decode_stats(const void* logits, const dllm_shape* shape, const uint8_t* masked,
                              const dllm_stats* out, void* ws, dllm_stream_t stream);

/*
 * Sampling (dInfer explainer, decoding strategies: a strategy takes each position's token and the
 * model's confidence in it): one token per row, drawn from the row's filtered softmax with a given
 * uniform number, in place of the most probable one.  For a computed row z of maximum m:
 *   candidates are ordered by falling z, lower ids first among equals, with weight
 *   w_v = exp((z_v - m) / temperature); each filter keeps a prefix of that order:
 *     top_k:  the first top_k (0, or V and more: all);
 *     top_p:  the shortest prefix that weighs at least top_p of what top_k keeps (1: all);
 *     min_p:  those with w_v >= min_p, that is z_v >= m + temperature * ln(min_p) (0: all);
 *   of the shortest of these prefixes the token is the lowest id at which the sum of the kept
 *   weights by rising id exceeds uniform[r] times their sum;
 *   row_max and lse as dllm_decode_stats;  argmax = the token;  conf = exp(z_token - lse), its
 *   probability under the model itself (no temperature, no filter).
 * The commit calls take these statistics with logits = NULL and so commit sampled tokens.
 * temperature 0 takes the most probable token (lowest id on ties), whatever the other fields.
 * A weight is off by at most 2^-36 of itself and half of 2^-42, and counts as 0 below 2^-42; weights
 * are summed exactly, so the token does not depend on how the work was split.  Rows with
 * masked[r] = 0 are not read and get -inf, -inf, 0, -1; so does a row without a finite logit, its lse
 * and row_max being what they are.
 * masked: [B*L] uint8 or NULL (every row).  uniform: [B*L] fp32 in [0, 1) (others count as the
 * nearest in range, a NaN as 0).  temperature 0 or in [2^-10, 2^10]; top_k >= 0; 0 < top_p <= 1;
 * 0 <= min_p <= 1; V <= 2^20.  Logits are finite or -inf.  No workspace.
 */
typedef struct {
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
} dllm_sampling;
dllm_status dllm_sample(const void* logits, const dllm_shape* shape, const uint8_t* masked,
                        const float* uniform, const dllm_sampling* how, const dllm_stats* out,
                        dllm_stream_t stream);

/*
 * Threshold decoding (dInfer explainer, decoding strategies, method 1: fix a position at once
 * when the model is confident in it).  Per sequence that is not stopped:
 *   C = { masked i : conf_i > tau };  if C is empty, C = { the masked i of largest conf,
 *   lowest i on ties };  for i in C: tokens[i] = argmax_i, masked[i] = 0, committed_now[i] = 1.
 * With logits != NULL the statistics are computed in the same pass (only the masked rows of
 * running sequences are read) and written to *stats; with logits == NULL, *stats must hold
 * the statistics of this step (conf and argmax are read) and the call only commits.
 * eos_id >= 0 enables the early stop; -1 disables it.
 */
dllm_status dllm_commit_threshold(const void* logits, const dllm_shape* shape,
                                  const dllm_stats* stats, const dllm_block_state* state,
                                  float tau, int32_t eos_id, void* ws, dllm_stream_t stream);

/*
 * Hierarchical decoding (dInfer explainer, decoding strategies, method 2: split the region
 * still to be filled recursively and decide the centre of each sub-region first).  Per
 * sequence that is not stopped, on the mask as it stands at the call:
 *   maximal runs [s, e) of masked positions are halved at s + floor(w/2) while their width
 *   w >= 2*min_width; in each resulting leaf the position with conf >= tau_low that is closest
 *   to the leaf centre (smallest |2i - (s+e-1)|, lowest i on ties) is committed; a sequence
 *   that commits nothing commits its masked position of largest conf (lowest i on ties).
 * min_width >= 1.  logits, stats, state and eos_id as in dllm_commit_threshold.
 */
dllm_status dllm_commit_hierarchical(const void* logits, const dllm_shape* shape,
                                     const dllm_stats* stats, const dllm_block_state* state,
                                     float tau_low, int32_t min_width, int32_t eos_id, void* ws,
                                     dllm_stream_t stream);

/*
 * Credit decoding (dInfer explainer, decoding strategies, method 3: each candidate token of
 * each position keeps a credit recording how often and how confidently it was chosen across
 * iterations; stable candidates are favoured).  Per masked position of a running sequence,
 * with top token a and confidence p:
 *   every slot decays, c_k <- decay*c_k;  a's slot gains p (a takes the first empty slot, or
 *   evicts the slot of least credit, lowest slot on ties, starting at p);
 *   score = p * (1 + boost * ln(1 + c_a));
 *   C = { i : score_i > tau }, or the masked i of largest score (lowest i) if C is empty.
 * cand_id: [B*L, K] int32 (-1 = empty slot), cand_credit: [B*L, K] fp32, both read and
 * updated; initialise to -1 / 0 for a fresh block.  Positions not masked keep their slots.
 * 1 <= K <= 16.
 */
dllm_status dllm_commit_credit(const void* logits, const dllm_shape* shape,
                               const dllm_stats* stats, const dllm_block_state* state,
                               int32_t* cand_id, float* cand_credit, int32_t K, float decay,
                               float boost, float tau, int32_t eos_id, void* ws,
                               dllm_stream_t stream);

/*
 * Hierarchical decoding, a centre per level (variant of dllm_commit_hierarchical; the pages'
 * "decide the centre of each sub-region first" read as deciding every level's centre).  Same
 * halving tree; every node [s, e), internal or leaf, selects its position with
 * conf >= tau_low closest to the node centre (smallest |2i - (s+e-1)|, lowest i on ties) and
 * the union of the selections is committed; fallback, arguments and errors as
 * dllm_commit_hierarchical.
 */
dllm_status dllm_commit_hierarchical_levels(const void* logits, const dllm_shape* shape,
                                            const dllm_stats* stats,
                                            const dllm_block_state* state, float tau_low,
                                            int32_t min_width, int32_t eos_id, void* ws,
                                            dllm_stream_t stream);

/*
 * Credit decoding, every tracked candidate credited (variant of dllm_commit_credit; dInfer
 * explainer, decoding strategies, method 3).  Per masked position of a running sequence, with
 * p_v = exp(z_v - lse), top token a and p_a = conf:
 *   every slot decays, c_k <- decay*c_k;  every occupied slot gains its own token's probability,
 *   c_k <- c_k + p_{id_k};  if a is not tracked it takes the first empty slot, or evicts the
 *   slot of least credit (after the gains; lowest slot on ties), starting at p_a;
 *   s_k = p_{id_k} * (1 + boost * ln(1 + c_k)) over occupied slots; the best slot (lowest slot on
 *   ties) is the position's candidate: score = s_k, token = id_k (may differ from a);
 *   C = { i : score_i > tau }, or the masked i of largest score (lowest i); commits the
 *   candidate tokens.
 * logits must not be NULL (the tracked tokens' logits are read after the statistics).  Other
 * arguments and errors as dllm_commit_credit.
 */
dllm_status dllm_commit_credit_tracked(const void* logits, const dllm_shape* shape,
                                       const dllm_stats* stats, const dllm_block_state* state,
                                       int32_t* cand_id, float* cand_credit, int32_t K,
                                       float decay, float boost, float tau, int32_t eos_id,
                                       void* ws, dllm_stream_t stream);

/*
 * Re-lay the embedding table once for the smoothing GEMM: E [V, d] bf16 row-major (the usual
 * table) -> Et, the transpose stored K-slab-blocked: Et[(v / 64) * d + c][v % 64] = E[v][c], so
 * that each 64-wide slab of the vocabulary is contiguous for every column c; slab entries with
 * v >= V are zero.  dllm_embedding_t_elems(V, d) = d * (V rounded up to 64) elements.  Bit
 * patterns are copied unchanged.  d % 16 == 0.  Et must be 16-byte aligned.
 */
size_t dllm_embedding_t_elems(int32_t V, int32_t d);
dllm_status dllm_prepare_embedding(const uint16_t* E, int32_t V, int32_t d, uint16_t* Et,
                                   dllm_stream_t stream);

/* Bytes of workspace dllm_smooth_embed needs (status word, bf16 probability rows, partials). */
size_t dllm_smooth_workspace_bytes(const dllm_shape* shape, int32_t d);

/*
 * How dllm_smooth_gemm will run on the current device (host query, launches nothing):
 * info[0] row tiles, info[1] column tiles, info[2] widest column tile, info[3] K ranges summed
 * per output element (1: the GEMM writes the output itself; more: split-K partial sums added by
 * a second kernel),
 * info[4] pipeline stages, info[5] kernels launched by one dllm_smooth_embed call.
 */
dllm_status dllm_smooth_plan_info(const dllm_shape* shape, int32_t d, int32_t* info);

/*
 * Iteration smoothing (dInfer explainer, diffusion-iteration manager: positions that stay
 * undecided keep their whole distribution for the next round instead of dropping it).  After
 * this step's commit, the rows still masked in sequences that are not stopped are listed in
 * ascending order, row_ids[0..M), and for each
 *   P[j, v] = bf16_round_nearest_even( exp(z_{row_ids[j], v} - lse_{row_ids[j]}) ),
 *   out[j, :] = sum_v P[j, v] * E[v, :]       (fp32 accumulation, tensor cores)
 * logits/shape: the step's logits (bf16 or fp32); stats: its statistics (lse is read);
 * state: the block state after the commit (masked, eos_hit read);
 * Et: the table from dllm_prepare_embedding; d % 16 == 0, d <= 65536;
 * out: [B*L, d] fp32, rows >= M untouched; row_ids: [B*L] int32, entries >= M set to -1;
 * M: one int32.  M is produced on the device; nothing is read back to the host.
 * ws: dllm_smooth_workspace_bytes(shape, d) bytes.  Logits rows that are not 16-byte aligned,
 * or V not a multiple of 8, are read element by element (same results).
 */
dllm_status dllm_smooth_embed(const void* logits, const dllm_shape* shape, const dllm_stats* stats,
                              const dllm_block_state* state, const uint16_t* Et, int32_t d,
                              float* out, int32_t* row_ids, int32_t* M, void* ws,
                              size_t ws_bytes, dllm_stream_t stream);

/*
 * The two halves of dllm_smooth_embed, for callers that schedule them separately (same
 * arguments and results; call them in this order on one stream with the same workspace):
 *   dllm_smooth_probs: rows kept (row_ids, M) and the bf16 probability rows P, written to the
 *                      workspace;
 *   dllm_smooth_gemm:  out[0..M) = P x E on the tensor cores.
 */
dllm_status dllm_smooth_probs(const void* logits, const dllm_shape* shape, const dllm_stats* stats,
                              const dllm_block_state* state, int32_t d, int32_t* row_ids,
                              int32_t* M, void* ws, size_t ws_bytes, dllm_stream_t stream);
dllm_status dllm_smooth_gemm(const dllm_shape* shape, const uint16_t* Et, int32_t d, float* out,
                             const int32_t* M, void* ws, size_t ws_bytes, dllm_stream_t stream);

/*
 * Statistics of rows whose vocabulary is split over n tensor-parallel shards (dInfer explainer,
 * system optimisations: tensor parallelism splits the output layer, so each GPU holds the logits
 * of one contiguous vocabulary range).  Shard k covers ids [vocab_offset, vocab_offset + V_k)
 * and its `stats` are dllm_decode_stats of those columns (local argmax).  Per row:
 *   row_max = max_k m_k;  s = sum_k exp(lse_k - row_max);  lse = row_max + ln s;  conf = 1/s;
 *   argmax = lowest vocab_offset_k + argmax_k over the shards with m_k = row_max.
 * A row that no shard read (all m_k = -inf) gets -inf, -inf, 0, -1.  Exchanging the shards'
 * statistics (R x 16 bytes each, an all-gather) is the caller's: `shards` is a host array of n
 * descriptors whose arrays are device memory on this GPU (this rank's own, or received).
 * n in [1, DLLM_MAX_SHARDS]; rows >= 0; out may not alias a shard's arrays.  Asynchronous on
 * `stream`; nothing is allocated.
 */
#define DLLM_MAX_SHARDS 64
typedef struct {
  dllm_stats stats;
  int64_t vocab_offset;
} dllm_shard_stats;
dllm_status dllm_merge_shard_stats(const dllm_shard_stats* shards, int32_t n, int64_t rows,
                                   const dllm_stats* out, dllm_stream_t stream);

/*
 * Threshold commit and iteration smoothing in one call, reading each logit from HBM once
 * (single-read smoothing).  Results are those of dllm_commit_threshold followed by
 * dllm_smooth_embed on the same arguments: the statistics of the rows read, the commit, and
 * out[0..M) = P x E for the rows kept (row_ids ascending, M on the device), within the same
 * tolerances.  The rows read are held on chip (a cluster of up to 8 CTAs per row, up to 192 KB
 * per CTA) while their log-sum-exp completes, so their probabilities are written without a
 * second read; the GEMM then covers the rows read (rows committed in this step included) and
 * writes only the kept ones.
 * ws: dllm_smooth_workspace_bytes(shape, d) bytes; Et prepared by dllm_prepare_embedding.
 * Rows the single-read kernels cannot hold whole (not 16-byte aligned, V not a multiple of 8, or
 * longer than 8 x 192 KB) give the same results through the separate calls (dllm_commit_threshold
 * then dllm_smooth_embed, which read rows that are not aligned element by element); the logits
 * are then read twice.
 */
dllm_status dllm_commit_threshold_smooth(const void* logits, const dllm_shape* shape,
                                        const dllm_stats* stats, const dllm_block_state* state,
                                        float tau, int32_t eos_id, const uint16_t* Et, int32_t d,
                                        float* out, int32_t* row_ids, int32_t* M, void* ws,
                                        size_t ws_bytes, dllm_stream_t stream);

/*
 * Neighbourhood KV refresh (dInfer explainer, KV-cache manager: when a region of the sequence
 * changes, its cache entries and those of its neighbours are recomputed).  The cache row of
 * sequence b is [prefix 0..prefix_len) followed by the block, T = prefix_len + L entries:
 *   refresh[b, j] = 1 iff some i with committed_now[b, i] = 1 has |j - (prefix_len + i)| <= window;
 *   idx[b, 0..count[b]) = the refreshed j ascending, idx[b, k] = -1 for k >= count[b].
 * refresh: [B, T] uint8; idx: [B, T] int32; count: [B] int32.  T <= 65536.
 */
dllm_status dllm_kv_refresh_mask(const dllm_block_state* state, int32_t B, int32_t L,
                                 int32_t prefix_len, int32_t window, uint8_t* refresh,
                                 int32_t* idx, int32_t* count, dllm_stream_t stream);

/*
 * Device-side early stop for decode loops captured as CUDA graphs (dInfer explainer, system
 * optimisations: the iterations run back to back on the GPU without waiting on the host, and
 * decoding stops as soon as the end token is produced instead of running the remaining
 * iterations).  A caller that captures its whole loop as one graph tests the block every k
 * iterations and captures the rest of the loop inside a conditional section on that test,
 * each section nested in the one before:
 *
 *   on S0 (capturing):  reset; iterations 0 .. k-1;
 *                       dllm_capture_condition(S0, 0, &h1); dllm_loop_continue(state, B, L, h1, S0);
 *                       dllm_capture_if_begin(S0, S1, h1);
 *     on S1:              iterations k .. 2k-1; the same test and a section on S2; ...
 *   innermost first:    dllm_capture_if_end(S_n); ... dllm_capture_if_end(S1);
 *
 * Once every sequence has stopped, the next test skips everything after it.  A conditional
 * section costs several microseconds of graph scheduling whether it runs or not (on a GB300:
 * ~8 us when taken, ~5 us when not, against ~1.4 us per plain kernel node), so a test every
 * few iterations, not every iteration, pays for itself.
 *
 * dllm_capture_condition: `stream` is capturing a CUDA graph (cudaStreamBeginCapture, directly
 * or through a framework).  Creates a condition handle in that graph with `default_value` (0 or
 * non-zero -> 1), assigned again at every launch of the graph.  *handle_out receives it.
 *
 * dllm_capture_if_begin: adds to the graph `stream` is capturing a conditional IF node on
 * `handle` (created by dllm_capture_condition on the same capture) that depends on everything
 * captured on `stream` so far, makes the node `stream`'s only capture dependency (later work
 * captured on `stream` runs after it) and starts capturing body_stream, another stream that is
 * not capturing, into the node's body: work enqueued on body_stream until dllm_capture_if_end
 * runs only when the handle is non-zero when the node is reached.  Sections nest: `stream` may
 * itself be a body stream.
 *
 * dllm_capture_if_end: ends the capture of a body begun by dllm_capture_if_begin (the body graph
 * belongs to the conditional node).
 *
 * dllm_loop_continue: captured in the graph that owns `handle` (at any depth of its conditional
 * sections); when the graph runs, sets the handle to 1 if some sequence b of the block still
 * decodes (eos_hit[b] = 0 and a masked position), else 0.  One CTA, ordered after the calls
 * before it on `stream`.  B >= 1, 1 <= L <= 1024, B*L <= 2^20.
 *
 * Errors: DLLM_ERR_INVALID_ARG (a null pointer, stream == body_stream, a stream that must be
 * capturing and is not, a body_stream already capturing); DLLM_ERR_CUDA (the driver refused the
 * handle or node, or the body capture was invalidated).  A handle that belongs to another graph
 * is not detected and must not be passed.
 */
dllm_status dllm_capture_condition(dllm_stream_t stream, uint32_t default_value,
                                   uint64_t* handle_out);
dllm_status dllm_capture_if_begin(dllm_stream_t stream, dllm_stream_t body_stream,
                                  uint64_t handle);
dllm_status dllm_capture_if_end(dllm_stream_t body_stream);
dllm_status dllm_loop_continue(const dllm_block_state* state, int32_t B, int32_t L,
                               uint64_t handle, dllm_stream_t stream);

/*
 * What a refresh runs through (dInfer explainer, KV-cache manager: the entries of a changed region
 * and its neighbours are recomputed).  dllm_kv_refresh_mask lists the entries; their new keys (and
 * the block's queries) are normalised per head and rotated to their positions
 * (dllm_qk_norm_rope), keys and values are stored in a cache of 4-bit codes (dllm_kv4_write) and
 * the block's queries attend over that cache (dllm_attention_kv4).  The index list of
 * dllm_kv_refresh_mask serves as `pos` of the calls below as it is: entries of -1 are skipped.
 *
 * dllm_heads describes rows of heads: channel c of head h of token i of sequence b is element
 *   data[b*batch_stride + i*token_stride + h*head_stride + c]
 * (strides in elements, so queries, keys and values may be slices of one projection's output).
 * Any strides and any pointer aligned to the element size are accepted; rows that all start on
 * 32-byte boundaries are read and written with wide accesses (16-byte boundaries do for
 * dllm_qk_norm_rope and dllm_attention_kv4), others element by element.
 */
typedef struct {
  void* data;
  int32_t heads;
  int32_t dtype; /* dllm_dtype */
  int64_t batch_stride;
  int64_t token_stride;
  int64_t head_stride;
} dllm_heads;

/*
 * Rotary frequencies: pair i of rotary_dim / 2 turns by f_i radians per position,
 *   g_i = base^(-2i / rotary_dim),
 *   DLLM_ROPE_LINEAR: f_i = g_i / factor  (factor 1: no scaling);
 *   DLLM_ROPE_BANDS:  with r_i = original_len * g_i / 2pi, the turns of pair i over the original
 *     context, and w = clamp((r_i - slow_turns) / (fast_turns - slow_turns), 0, 1):
 *     f_i = (1 - w) * g_i / factor + w * g_i   (pairs that turn often keep their frequency, slow
 *     ones are interpolated: the "by parts" rule of the YaRN paper, arXiv 2309.00071, section 3.2).
 * dllm_rope_phases writes phases[i] = round(f_i / 2pi * 2^64), rotary_dim / 2 device words: the
 * fraction of a turn per position in units of 2^-64, so that position * phases[i] modulo 2^64 is
 * the phase without a loss at long positions.  Run it once per model.  rotary_dim even,
 * 2 <= rotary_dim <= 1024; base > 1; factor >= 1; for BANDS original_len > 0 and
 * 0 <= slow_turns < fast_turns.
 */
typedef enum { DLLM_ROPE_LINEAR = 0, DLLM_ROPE_BANDS = 1 } dllm_rope_scaling;
typedef struct {
  int32_t rotary_dim;
  int32_t scaling; /* dllm_rope_scaling */
  double base;
  double factor;
  double original_len;
  double slow_turns;
  double fast_turns;
} dllm_rope;
dllm_status dllm_rope_phases(const dllm_rope* rope, int64_t* phases, dllm_stream_t stream);

/*
 * Norm of each head of queries and keys and rotation to the token's position, in one pass.  Per
 * token (b, i) with p = pos[b*pos_stride + i] >= 0 (tokens with p < 0 are skipped: their output
 * is left as it is), per head x of head_dim channels:
 *   y = norm ? x * (mean(x^2) + eps)^(-1/2) * weight : x       (weight NULL: ones)
 *   each pair (a, c) = (y[i], y[i + rotary_dim/2]) or, interleaved, (y[2i], y[2i+1]), i <
 *   rotary_dim/2:  (a cos t - c sin t, c cos t + a sin t) * magnitude,  t = 2pi * p*phases[i]/2^64;
 *   the other channels are y.
 * All in fp32, rounded once to the output.  q and q_out (k and k_out) have the same number of
 * heads; they may be the same memory with the same strides, and must not overlap otherwise.
 * q, q_out or k, k_out may be NULL (both of a pair): only the other is done.  One dtype for all
 * tensors and weights (fp32 or bf16).  1 <= head_dim <= 1024; rotary_dim even, <= head_dim, 0: no
 * rotation (phases may be NULL, and pos too: every token is done).  B, n >= 1, B*n <= 2^20, and
 * B*n times the heads of q and k together <= 2^33 - 4.
 */
dllm_status dllm_qk_norm_rope(const dllm_heads* q, const dllm_heads* q_out, const dllm_heads* k,
                              const dllm_heads* k_out, int32_t B, int32_t n, int32_t head_dim,
                              const int32_t* pos, int64_t pos_stride, const int64_t* phases,
                              int32_t rotary_dim, int32_t interleaved, float magnitude,
                              int32_t norm, const void* q_weight, const void* k_weight, float eps,
                              dllm_stream_t stream);

/*
 * A cache of keys and values in 4-bit codes, in pages.  Entry p of sequence b is slot
 * p % page_size of page page_table[b*table_stride + p / page_size]; a table word outside
 * [0, pages) means that the page is absent.  32 channels of one entry of one head are a group with
 * a step s (fp32 value with three significant bits) and a zero point z in 0..15; code n stands
 * for s * (n - z), which bf16 holds exactly.  codes: [pages, heads, page_size, head_dim / 2]
 * bytes, channel 2c in the low nibble of byte c.  params: [pages, heads, page_size, head_dim / 32]
 * 16-bit words, the bf16 bits of s with z in the low four.  4.5 bits a value.
 * heads <= 4096; page_size a multiple of 16 in [16, 65536]; head_dim a multiple of 32 in [32, 512];
 * codes and params 16-byte aligned.  The caller owns all arrays; nothing has to be initialised.
 */
typedef struct {
  uint8_t* k_codes;
  uint16_t* k_params;
  uint8_t* v_codes;
  uint16_t* v_params;
  const int32_t* page_table;
  int32_t pages;
  int32_t heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t table_stride; /* words (pages) of a sequence in page_table */
} dllm_kv4_cache;

/*
 * Quantise keys and values as they are written: token (b, i) goes to entry pos[b*pos_stride + i]
 * of sequence b.  Entries < 0, beyond the page table or on an absent page are skipped; the entries
 * of one call must differ from each other.  Per group x of 32 channels, in fp32:
 *   lo = min(0, min x), hi = max(0, max x), s = (hi - lo) / 15 rounded up to three significant
 *   bits (0 if below 2^-110), z = floor(-lo / s + 1/2),
 *   n = min(15, round(x / s) + z), round half away from zero: |x - s (n - z)| <= s / 2.
 * A group that holds a NaN or an infinity, or whose s exceeds 2^122, reads back as NaN.
 * k, v: cache->heads heads, one dtype (fp32 or bf16).  B, n >= 1, B*n <= 2^20.
 */
dllm_status dllm_kv4_write(const dllm_kv4_cache* cache, const dllm_heads* k, const dllm_heads* v,
                           int32_t B, int32_t n, const int32_t* pos, int64_t pos_stride,
                           dllm_stream_t stream);

/*
 * Read entries back: k and v of token (b, i) receive the values of entry pos[b*pos_stride + i]
 * (pos NULL: entry i), exact in both dtypes; entries < 0, beyond the table or on an absent page
 * read as 0.  Limits as dllm_kv4_write.
 */
dllm_status dllm_kv4_read(const dllm_kv4_cache* cache, const dllm_heads* k, const dllm_heads* v,
                          int32_t B, int32_t n, const int32_t* pos, int64_t pos_stride,
                          dllm_stream_t stream);

/*
 * Attention of n queries per sequence over the cache (a block of positions being decoded, a single
 * token, a piece of a prompt).  Query head h reads key/value head h / (q->heads / cache->heads).
 * Query i of sequence b sees entry j when
 *   j < len_b = min(lens[b], max_len)  (lens NULL: max_len),  key_mask[b*mask_stride + j] != 0
 *   (key_mask NULL: all; mask_stride >= max_len, or 0: one mask for all sequences),  its page is
 *   present, and, with `causal`, j <= len_b - n + i;
 *   lse = ln sum_j exp(scale * q.K_j),  out = sum_j exp(scale * q.K_j - lse) V_j.
 * A query that sees nothing gets out = 0 and lse = -inf.  Entries that a query does not see have no
 * effect on it, whatever their codes, params and mask neighbours hold.  A score that is NaN makes
 * out and lse of its query NaN, a group of V that reads as NaN its 32 channels of every query that
 * sees the entry.  Scores, the softmax statistics and sums are fp32; the weights exp(.) are rounded
 * to bf16 for their product with V, which is exact bf16, and out is rounded once to bf16.  The order
 * of all sums is fixed: repeated calls agree bit for bit.
 * q, out: bf16, same heads (a multiple of cache->heads); they may be the same memory with the same
 * strides, and must not overlap otherwise.  lse: [B, q->heads, n] fp32 or NULL.
 * head_dim 64, 128, 192 or 256; 0 <= max_len <= table_stride * page_size and 2^30; scale finite;
 * B*n <= 2^20, B*n*heads <= 2^30.
 * ws: dllm_attention_kv4_workspace_bytes(...) bytes (0 on invalid sizes); max_len is the bound the
 * split of the entries over the GPU is planned from, lens are read on the device.
 */
size_t dllm_attention_kv4_workspace_bytes(const dllm_kv4_cache* cache, int32_t B, int32_t n,
                                          int32_t q_heads, int32_t max_len);
dllm_status dllm_attention_kv4(const dllm_heads* q, const dllm_kv4_cache* cache,
                               const int32_t* lens, int32_t max_len, const uint8_t* key_mask,
                               int64_t mask_stride, float scale, int32_t causal,
                               const dllm_heads* out, float* lse, int32_t B, int32_t n, void* ws,
                               size_t ws_bytes, dllm_stream_t stream);

/*
 * How much attention each cache entry receives from the queries of one dllm_attention_kv4 call, added
 * to what earlier calls left (dInfer explainer, KV-cache manager: which entries a cache keeps).  For
 * j < len_b:
 *   weights[b, j] = keep * prior[b, j] + sum over queries i and heads h that see j of
 *                   exp(scale * q_ih.K_j - lse_ih)
 * with the visibility, q, cache, lens, key_mask, scale and causal of that call and the lse it wrote.
 * weights and prior: fp32, row b from b * their stride on (strides >= max_len); they may be the same
 * memory with the same stride, and must not overlap otherwise; prior NULL: nothing is added, and keep
 * is not used.  Words of weights from len_b on are left as they are.  A query whose lse is -inf saw
 * nothing and adds nothing, one whose lse is +inf adds 0 by the formula; a score that is NaN makes the
 * weight of its entry NaN, a NaN of lse those of all entries its query sees.  All in fp32, in a fixed order: repeated calls agree bit for bit.
 * Limits as dllm_attention_kv4, and B * max_len <= 2^36.
 * ws: dllm_attention_kv4_weights_workspace_bytes(...) bytes (0 on invalid sizes).
 */
size_t dllm_attention_kv4_weights_workspace_bytes(const dllm_kv4_cache* cache, int32_t B, int32_t n,
                                                  int32_t q_heads, int32_t max_len);
dllm_status dllm_attention_kv4_weights(const dllm_heads* q, const dllm_kv4_cache* cache,
                                       const int32_t* lens, int32_t max_len,
                                       const uint8_t* key_mask, int64_t mask_stride, float scale,
                                       int32_t causal, const float* lse, const float* prior,
                                       int64_t prior_stride, float keep, float* weights,
                                       int64_t weights_stride, int32_t B, int32_t n, void* ws,
                                       size_t ws_bytes, dllm_stream_t stream);

/*
 * Eviction (dInfer explainer, KV-cache manager): cut every sequence to at most `budget` entries, by
 * the weights that dllm_attention_kv4_weights adds up.  With len_b = min(lens[b], max_len) (lens NULL:
 * max_len) and new_b = min(len_b, budget), a sequence of more than `budget` entries keeps its first
 * `first` and last `last` entries and, of the others, those of largest weight (lower entries first
 * among equals; a NaN is less than every number), new_b in all.  Kept entries before new_b stay where
 * they are; the k-th kept entry from new_b on moves to the place of the k-th dropped entry before
 * new_b, codes and params of all heads.  Attention does not depend on the order of entries: keys hold
 * their rotation.  (A `causal` call does: it takes the last n entries for its queries'.  Write those
 * after an eviction.)
 *   slots[b*slots_stride + j], j < max_len: where entry j is now, -1 if it was dropped or j >= len_b
 *     (a list of positions goes through it before dllm_kv4_write);
 *   lens_out[b] = new_b; it may be lens;
 *   weights_out (or NULL), j < max_len: the weights in the entries' new order, 0 from new_b on; it may
 *     be weights with the same stride, and must not overlap it otherwise.
 * Entries from new_b on and pages are left as they are; pages wholly behind new_b may be reused.  The
 * pages of a sequence's first len_b entries must be its own; a move from or to an absent page is not
 * made.  budget, first, last >= 0, first + last <= budget; 0 <= max_len <= table_stride * page_size
 * and 2^30; B >= 1, B <= 2^20, B * max_len <= 2^36; strides >= max_len.
 * ws: dllm_kv4_evict_workspace_bytes(cache, B, max_len) bytes (0 on invalid sizes).
 */
size_t dllm_kv4_evict_workspace_bytes(const dllm_kv4_cache* cache, int32_t B, int32_t max_len);
dllm_status dllm_kv4_evict(const dllm_kv4_cache* cache, const float* weights, int64_t weights_stride,
                           const int32_t* lens, int32_t max_len, int32_t budget, int32_t first,
                           int32_t last, int32_t* slots, int64_t slots_stride, int32_t* lens_out,
                           float* weights_out, int64_t weights_out_stride, int32_t B, void* ws,
                           size_t ws_bytes, dllm_stream_t stream);

/*
 * Self-test of failure detection (no counterpart in the pages): runs the bounded wait the
 * smoothing GEMM uses on a barrier that nothing ever completes.  After limit_us microseconds
 * (1 .. 2,000,000) the wait gives up and records DLLM_ERR_TIMEOUT in the status word of `ws`
 * (any workspace, or 256 zeroed bytes); read it with dllm_get_status.  Nothing faults or hangs.
 */
dllm_status dllm_selftest_wait_timeout(void* ws, uint32_t limit_us, dllm_stream_t stream);

/*
 * dllm_commit_threshold without a workspace argument, for callers that cannot allocate device
 * memory where they decode (a serving runtime that reserves all memory up front and forbids
 * allocation while requests are in flight, a plugin whose host framework owns every device
 * buffer).  The pages have no counterpart to this call; it exists for those callers only.
 * Same arguments (minus ws), same results and same errors as dllm_commit_threshold with
 * logits != NULL, computed by the same kernel.  Its scratch is one static array of
 * DLLM_STATIC_WORKSPACE_BYTES in device memory, part of the library image: every GPU that loads
 * the library holds it until the process exits.
 *  - Shapes whose dllm_workspace_bytes exceeds DLLM_STATIC_WORKSPACE_BYTES are rejected with
 *    DLLM_ERR_UNSUPPORTED (4 MiB: e.g. B*L up to 2048 rows at V = 126464).
 *  - The first call on a device looks up the array's device address (cudaGetSymbolAddress) with
 *    that device current; make that first call before any stream capture.
 *  - Each call clears the array's status word on `stream`; nothing is allocated or freed.
 *    All calls share the one array and it keeps the last call's contents, so calls that
 *    overlap on the GPU (different streams, or concurrent graphs) race: serialise them.
 *  - dllm_get_status cannot be used on this scratch; a fault inside the kernel still surfaces
 *    as wrong results only, as for any call whose status word is never read.
 */
#define DLLM_STATIC_WORKSPACE_BYTES ((size_t)4 << 20)
dllm_status dllm_commit_threshold_static(const void* logits, const dllm_shape* shape,
                                         const dllm_stats* stats, const dllm_block_state* state,
                                         float tau, int32_t eos_id, dllm_stream_t stream);

/*
 * Read the device status word of a workspace (its first 4 bytes; synchronises `stream`).
 * *out_host receives DLLM_OK or the first fault a kernel recorded there (DLLM_ERR_TIMEOUT);
 * the word is then reset to DLLM_OK.  Works for both kinds of workspace.
 */
dllm_status dllm_get_status(void* ws, dllm_stream_t stream, int32_t* out_host);

#ifdef __cplusplus
}
#endif

#endif /* DLLM_H_ */
