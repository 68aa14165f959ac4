// Device helpers of the accumulated attention weights.
#pragma once

#include "attention.h"
#include "common.cuh"

namespace dllm {

// -lse in the scores' units (base 2); -inf of +inf, by which a query adds 0.
__device__ __forceinline__ float minus_l(const AttnWeights& x, float lse) {
  const float l = lse == INFINITY ? 0x1.fffffep127f : lse;  // (its product is infinite)
  return -fmaf(l, x.l_hi, l * x.l_lo);
}
__device__ __forceinline__ void put_weight(const AttnWeights& x, int b, int j, float got) {
  x.out[b * x.out_stride + j] = x.prior ? fmaf(x.keep, x.prior[b * x.prior_stride + j], got) : got;
}

}  // namespace dllm
