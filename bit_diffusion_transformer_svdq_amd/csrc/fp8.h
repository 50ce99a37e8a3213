// Internal to the kernels of the 8-bit floating-point linear (e4m3 codes, a scale for
// each block of 128).
#pragma once

#include "row_device.h"
#include "w8a8.h"

namespace svdq {

constexpr int kFp8Block = 128;

// SiLU, x / (1 + exp(-x)): relative error below (1.23 |x| + 6) 2^-24 for x > -87 (the
// product with log2(e) is rounded, |x| of it, and log2(e) itself is off by 0.23 2^-24);
// beyond, where the reciprocal is subnormal and v_rcp_f32 gives zero, values below
// 1e-36 in magnitude come out as -0
__device__ __forceinline__ float silu_exp2(float x) {
  return x * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(-1.442695041f * x) + 1.0f);
}

__device__ __forceinline__ float gate_act(float g, int act) { return act == kActSilu ? silu_exp2(g) : gelu_exp2(g); }

// A block's scale and its reciprocal from its largest magnitude: s = fl32(A fl32(1/448)),
// 448 the largest e4m3 value.  A block whose 1/s is not finite (A = 0, or below about
// 1.3e-36) gets codes 0, one with an infinity or NaN codes 0 and s = NaN, so that its
// products are NaN.
__device__ __forceinline__ void block_scale(float amax, float& s, float& inv) {
  s = amax * (1.0f / 448.0f);
  inv = rcp_is_plain(s) ? rcp_plain(s) : 1.0f / s;
  if (!(inv < __builtin_inff())) inv = 0.0f;
  if (!(amax < __builtin_inff())) {
    s = __builtin_nanf("");
    inv = 0.0f;
  }
}

// four e4m3 codes of fl32(v inv), nearest even; |v| inv <= 448 (1 + 2^-22) rounds to
// 448 at most.  An infinity or NaN times inv = 0 is masked by the caller.
__device__ __forceinline__ row_u32 fp8_codes4(const float* v, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  return (row_u32)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
}

// maximum over each 16 lanes
__device__ __forceinline__ float max16(float x) {
  x = BitMaxOp::run(x, dpp_mov<0x128>(x));
  x = BitMaxOp::run(x, dpp_mov<0x124>(x));
  x = BitMaxOp::run(x, dpp_mov<0x122>(x));
  return BitMaxOp::run(x, dpp_mov<0x121>(x));
}
// over the four lanes l, l + 16, l + 32, l + 48
__device__ __forceinline__ float max_rows4(float x) {
  const row_u32 u = __builtin_bit_cast(row_u32, x);
  const auto s16 = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = BitMaxOp::run(__builtin_bit_cast(float, (row_u32)s16[0]), __builtin_bit_cast(float, (row_u32)s16[1]));
  const row_u32 w = __builtin_bit_cast(row_u32, x);
  const auto s32 = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return BitMaxOp::run(__builtin_bit_cast(float, (row_u32)s32[0]), __builtin_bit_cast(float, (row_u32)s32[1]));
}

// up to 16 tokens: the weight-streaming kernel
size_t fp8_skinny_workspace_bytes(const Fp8Args& a);
hipError_t launch_fp8_skinny(const Fp8Args& a, Workspace ws, hipStream_t stream);

}  // namespace svdq
