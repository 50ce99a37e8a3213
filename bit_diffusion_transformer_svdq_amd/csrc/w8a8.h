// Internal to the 8-bit linear's kernels.
#pragma once

#include "row_device.h"

namespace svdq {

// GELU (tanh form), x (1 + tanh u) / 2 = x / (1 + exp(-2u)), exp(-2u) = 2^t with
// t = -x (c0 + c1 x^2): one exponential and one reciprocal, five other operations;
// the relative error stays below (3.5 |t| + 7) 2^-24 for t < 126 (x > -10).  Beyond,
// the reciprocal is subnormal, which v_rcp_f32 gives as zero: values below 1.2e-37 in
// magnitude come out as -0
__device__ __forceinline__ float gelu_exp2(float x) {
  constexpr float c0 = 2.302208198f, c1 = 0.1029432397f;  // 2 sqrt(2/pi) log2(e), and 0.044715 times it
  const float e = __builtin_amdgcn_exp2f(x * __builtin_fmaf(-c1, x * x, -c0));
  return x * __builtin_amdgcn_rcpf(e + 1.0f);
}

// up to 16 tokens: the weight-streaming kernel
hipError_t launch_w8a8_skinny(const W8a8Args& a, hipStream_t stream);

}  // namespace svdq
