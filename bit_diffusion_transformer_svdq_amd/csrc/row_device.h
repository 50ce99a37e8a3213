// Device helpers of the kernels that own one row per wave or workgroup.
#pragma once

#include "svdq_device.h"

namespace svdq {

typedef unsigned int row_u32;
typedef row_u32 row_v2u __attribute__((ext_vector_type(2)));
typedef row_u32 row_v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(row_u32 w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(row_u32 w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& p, float (&f)[8]) {
  f[0] = bf16_lo(p.x), f[1] = bf16_hi(p.x), f[2] = bf16_lo(p.y), f[3] = bf16_hi(p.y);
  f[4] = bf16_lo(p.z), f[5] = bf16_hi(p.z), f[6] = bf16_lo(p.w), f[7] = bf16_hi(p.w);
}

// two fp32 values to packed bf16, nearest even
__device__ __forceinline__ row_u32 pack2_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(row_u32, __builtin_convertvector(f2{a, b}, b2));
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return uint4{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7])};
}

struct SumOp {
  static __device__ __forceinline__ float run(float a, float b) { return a + b; }
};
// maximum of the bit patterns of non-negative floats: orders like the values,
// and a NaN is larger than infinity instead of being passed over
struct BitMaxOp {
  static __device__ __forceinline__ float run(float a, float b) {
    const row_u32 x = __builtin_bit_cast(row_u32, a), y = __builtin_bit_cast(row_u32, b);
    return __builtin_bit_cast(float, x > y ? x : y);
  }
};

template <int kCtrl>
__device__ __forceinline__ float dpp_mov(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), kCtrl, 0xF, 0xF, true));
}

// All-reduce over the 64 lanes: rotations by 8, 4, 2, 1 inside each row of 16
// lanes, then the lane swaps across rows and halves.  At every step the lanes
// that are combined hold equal operands in either order, so all lanes end
// with the same bits.
template <class Op>
__device__ __forceinline__ float wave_reduce(float x) {
  x = Op::run(x, dpp_mov<0x128>(x));  // row_ror:8
  x = Op::run(x, dpp_mov<0x124>(x));
  x = Op::run(x, dpp_mov<0x122>(x));
  x = Op::run(x, dpp_mov<0x121>(x));
  const row_u32 u = __builtin_bit_cast(row_u32, x);
  const auto s16 = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = Op::run(__builtin_bit_cast(float, (row_u32)s16[0]), __builtin_bit_cast(float, (row_u32)s16[1]));
  const row_u32 w = __builtin_bit_cast(row_u32, x);
  const auto s32 = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return Op::run(__builtin_bit_cast(float, (row_u32)s32[0]), __builtin_bit_cast(float, (row_u32)s32[1]));
}

// All-reduce over the W waves of a workgroup that owns one row: each wave's
// value meets the others' in LDS slot `slot` (a slot of its own per
// reduction, so one barrier is enough), in wave order.
template <class Op, int W>
__device__ __forceinline__ float row_reduce(float x, float* lds, int slot) {
  x = wave_reduce<Op>(x);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[slot * W + wave] = x;
    __syncthreads();
    x = lds[slot * W];
#pragma unroll
    for (int w = 1; w < W; ++w) x = Op::run(x, lds[slot * W + w]);
  }
  return x;
}

// fl32(1 / s), correctly rounded, in the place of s.  v_rcp_f32 is within one ulp,
// and one Newton step with an exact residual then rounds correctly except where
// every significand bit of s is one (Markstein, 1990); those, and exponents near
// the ends of the range, take the IEEE division.
__device__ __forceinline__ bool rcp_is_plain(float s) {
  const row_u32 b = __builtin_bit_cast(row_u32, s) & 0x7FFFFFFFu;
  return b >= (27u << 23) && b < (227u << 23) && (b & 0x7FFFFFu) != 0x7FFFFFu;
}
__device__ __forceinline__ float rcp_plain(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
}
__device__ __forceinline__ void recip8(float (&s)[8]) {
  bool plain = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) plain = plain && rcp_is_plain(s[e]);
  if (__all(plain)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = rcp_plain(s[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 1.0f / s[e];
  }
}

// The 8-bit token scale and its reciprocal from the row's largest magnitude:
// s = fl32(A / 127).  A row whose 1/s is not finite (A = 0, or below about
// 4e-37) gets codes 0, a row with an infinity or NaN codes 0 and s = NaN, so
// that its products are NaN.
__device__ __forceinline__ void token_scale(float amax, float& s, float& inv) {
  s = amax / 127.0f;
  inv = 1.0f / s;
  if (!(inv < __builtin_inff())) inv = 0.0f;
  if (!(amax < __builtin_inff())) {
    s = __builtin_nanf("");
    inv = 0.0f;
  }
}

// four codes rint(v * inv) in one word (the exact product, rounded once by the
// fma against 1.5 * 2^23, whose low byte is the code in two's complement).
// |v| inv <= 127 (1 + 2^-20), so no clamp is needed; a NaN or infinity times
// inv = 0 is masked by the caller.
__device__ __forceinline__ row_u32 codes4(const float* v, float inv) {
  row_u32 b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = __builtin_bit_cast(row_u32, __builtin_fmaf(v[e], inv, 12582912.0f));
  const row_u32 lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
  const row_u32 hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
  return lo | hi;
}

}  // namespace svdq
