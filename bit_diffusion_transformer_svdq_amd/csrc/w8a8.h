// Internal to the 8-bit linear's kernels.
#pragma once

#include "row_device.h"

namespace svdq {

// GELU (tanh form) as x - x / (exp(2u) + 1) with exp(2u) = 2^(x (c0 + c1 x^2)): one
// exponential and one reciprocal, five other operations; within 2^-21 |x|
__device__ __forceinline__ float gelu_exp2(float x) {
  constexpr float c0 = 2.302208198f, c1 = 0.1029432397f;  // 2 sqrt(2/pi) log2(e), and 0.044715 times it
  const float e = __builtin_amdgcn_exp2f(x * __builtin_fmaf(c1, x * x, c0));
  return __builtin_fmaf(-x, __builtin_amdgcn_rcpf(e + 1.0f), x);
}

// up to 16 tokens: the weight-streaming kernel
hipError_t launch_w8a8_skinny(const W8a8Args& a, hipStream_t stream);

}  // namespace svdq
