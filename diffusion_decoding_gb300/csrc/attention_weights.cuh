// Device helpers of the accumulated attention weights.
#pragma once

#include "attention.h"
#include "common.cuh"

namespace dllm {

// -lse in the scores' units (base 2).
__device__ __forceinline__ float minus_l(const AttnWeights& x, float lse) {
  return -fmaf(lse, x.l_hi, lse * x.l_lo);
}
__device__ __forceinline__ void put_weight(const AttnWeights& x, int b, int j, float got) {
  x.out[b * x.out_stride + j] = x.prior ? fmaf(x.keep, x.prior[b * x.prior_stride + j], got) : got;
}

}  // namespace dllm
