// Launch interface of the attention over the 4-bit cache.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dllm {

struct AttnParams {
  const uint16_t* q;  // strides in elements
  int64_t qb, qt, qh;
  uint16_t* out;
  int64_t ob, ot, oh;
  float* lse;  // [B, heads * G, n] or null
  const uint8_t* k_codes;
  const uint16_t* k_params;
  const uint8_t* v_codes;
  const uint16_t* v_params;
  const int32_t* table;
  int table_stride, pages, page_size;
  int heads;  // of the cache
  int G;      // query heads per cache head
  uint32_t g_magic;  // floor(2^32 / G) + 1: r / G = umulhi(r, g_magic) while r * G < 2^32 (0: divide)
  const int32_t* lens;
  int max_len;
  const uint8_t* key_mask;
  int64_t mask_stride;
  float scale_log2;  // scale * log2(e): scores are kept in base 2
  int causal;
  int B, n;
};

size_t attention_ws_bytes(int B, int n, int G, int heads, int D, int max_len, int sm_count);

cudaError_t launch_attention(const AttnParams& p, int D, void* ws, int sm_count, cudaStream_t stream);

// Many rows per cache head (attention_tc.cu): whether it can have these rows, and has this call.
bool attention_tc_can(int n, int G, int D);
bool attention_tc_takes(const AttnParams& p, int D, int sm_count);
size_t attention_tc_ws_bytes(int B, int n, int G, int heads, int D, int sm_count);
cudaError_t launch_attention_tc(const AttnParams& p, int D, void* ws, int sm_count,
                                cudaStream_t stream);

// Division of n < 2^31 by a number known on the host: a multiplication (of at most 2^32 / 2^l * (1 + 2^-31)
// for 2^(l-1) < d <= 2^l) and a shift.
struct Divisor {
  uint32_t d, m, shift;  // d = 1: m = 0
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return m ? __umulhi(n, m) >> shift : n; }
};
inline Divisor divisor(uint32_t d) {
  if (d <= 1) return Divisor{1u, 0u, 0u};
  uint32_t l = 1;
  while ((uint64_t{1} << l) < d) ++l;
  return Divisor{d, static_cast<uint32_t>(((uint64_t{1} << (31 + l)) + d - 1) / d), l - 1};
}

// Accumulated weights (attention_weights.cu): the call's queries, cache and masks are an AttnParams
// (out and lse unused).
struct AttnWeights {
  const float* lse;    // [B, heads * G, n]
  const float* prior;  // null: 0
  int64_t prior_stride;
  float* out;
  int64_t out_stride;
  float keep;
  float scale;
  float l_hi, l_lo;  // scale_log2 / scale: what a log-sum-exp is multiplied by
  int q_aligned;
  Divisor by_page;
  int ctas_per_seq, split_log2, heads_at_once, tiles_per_warp;  // few rows: attention_weights.cu
};
size_t attention_weights_ws_bytes(int B, int n, int G, int heads, int D, int max_len);
cudaError_t launch_attention_weights(const AttnParams& p, AttnWeights x, int D, void* ws, int sm_count,
                                     cudaStream_t stream);

// Many rows per cache head (attention_weights_tc.cu).
bool weights_tc_scale(float scale);  // whether it can have this scale
bool weights_tc_takes(int B, int n, int G, int heads, int D, int max_len);
size_t weights_tc_ws_bytes(int B, int n, int G, int heads, int D, int max_len);
cudaError_t launch_weights_tc(const AttnParams& p, const AttnWeights& x, int D, void* ws, int sm_count,
                              cudaStream_t stream);

// Rows of a bf16 tensor (strides in elements) all start on 16-byte boundaries.
bool attention_rows_aligned(const void* x, int64_t sb, int64_t st, int64_t sh);

}  // namespace dllm
