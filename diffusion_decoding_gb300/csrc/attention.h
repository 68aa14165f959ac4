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

// Rows of a bf16 tensor (strides in elements) all start on 16-byte boundaries.
bool attention_rows_aligned(const void* x, int64_t sb, int64_t st, int64_t sh);

}  // namespace dllm
