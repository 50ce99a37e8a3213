// The 8-bit linear for up to 64 tokens on gfx950: a weight stream.
//
// With few tokens the product is bound by reading the weights once (N K bytes).
// A workgroup owns 16 NT weight rows and its 8 waves divide K: each wave reads
// its part of the rows straight into registers (16 rows x 64 bytes per load
// instruction), the same part of the token rows from L2, and accumulates
// v_mfma_i32_16x16x64_i8 tiles.  The waves' int32 partial tiles are added in LDS.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_device.h"
#include "w8a8.h"

namespace svdq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// MT token tiles of 16, kDepth k steps of 64 in flight per wave
template <int NT, int MT, int kDepth>
__global__ __launch_bounds__(kThreads) void w8a8_skinny_kernel(const W8a8Args a) {
  __shared__ __attribute__((aligned(16))) v4i red[kWaves][NT * MT][64];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT;
  const int P = a.K >> 6;
  const int p0 = (int)((long)wave * P / kWaves), p1 = (int)((long)(wave + 1) * P / kWaves);

  const int8_t* wr[NT];
  const int8_t* ar[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) wr[j] = a.w + (size_t)min(n0 + 16 * j + l16, a.N - 1) * a.K + 16 * lq;
#pragma unroll
  for (int i = 0; i < MT; ++i) ar[i] = a.act + (size_t)min(16 * i + l16, a.M - 1) * a.K + 16 * lq;
  v4i acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = v4i{0, 0, 0, 0};

  v4i fw[kDepth][NT], fa[kDepth][MT];
  // steps past the wave's range repeat its last one (their products are not
  // added), so every load is unconditional
  auto fetch = [&](int s, int p) {
    const int off = 64 * max(0, min(p, p1 - 1));
#pragma unroll
    for (int j = 0; j < NT; ++j) fw[s][j] = *reinterpret_cast<const v4i*>(wr[j] + off);
#pragma unroll
    for (int i = 0; i < MT; ++i) fa[s][i] = *reinterpret_cast<const v4i*>(ar[i] + off);
  };
#pragma unroll
  for (int s = 0; s < kDepth; ++s) fetch(s, p0 + s);
  for (int p = p0; p < p1; p += kDepth) {
#pragma unroll
    for (int s = 0; s < kDepth; ++s) {
      if (p + s < p1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[s][j], fa[s][i], acc[j][i], 0, 0, 0);
      }
      fetch(s, p + s + kDepth);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][j * MT + i][lane] = acc[j][i];
  __syncthreads();
  for (int it = tid; it < NT * MT * 64; it += kThreads) {
    const int t = it >> 6, j = t / MT, i = t - j * MT;
    const int m = 16 * i + l16, n = n0 + 16 * j + 4 * lq;  // it % 64 == lane
    v4i s = red[0][t][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[w][t][lane];
    if (m < a.M && n < a.N) {  // N % 64 == 0
      const float sx = a.act_scales[m];
      const float4 sw = *reinterpret_cast<const float4*>(a.w_scales + n);
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      if (a.bias != nullptr) {
        const uint2 b2 = *reinterpret_cast<const uint2*>(a.bias + n);
        b[0] = bf16_lo(b2.x), b[1] = bf16_hi(b2.x), b[2] = bf16_lo(b2.y), b[3] = bf16_hi(b2.y);
      }
      float o[4] = {__builtin_fmaf((float)s[0], sx * sw.x, b[0]), __builtin_fmaf((float)s[1], sx * sw.y, b[1]),
                    __builtin_fmaf((float)s[2], sx * sw.z, b[2]), __builtin_fmaf((float)s[3], sx * sw.w, b[3])};
      if (a.epilogue == kEpilogueGelu) {
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = gelu_tanh(o[v]);
      }
      *reinterpret_cast<uint2*>(a.y + (size_t)m * a.N + n) = uint2{pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3])};
    }
  }
}

template <int NT, int MT>
void go(const W8a8Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((w8a8_skinny_kernel<NT, MT, 2>), dim3((a.N + 16 * NT - 1) / (16 * NT)), dim3(kThreads), 0, stream,
                     a);
}

}  // namespace

hipError_t launch_w8a8_skinny(const W8a8Args& a, hipStream_t stream) {
  if (a.M > 64) return hipErrorInvalidValue;
  const int n16 = a.N / 16;
  // as many rows per workgroup as keep every compute unit busy once
  const int nt = n16 >= 3 * current_cus() ? 3 : n16 >= 2 * current_cus() ? 2 : 1;
  const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  switch (10 * nt + mt) {
    case 11: go<1, 1>(a, stream); break;
    case 12: go<1, 2>(a, stream); break;
    case 14: go<1, 4>(a, stream); break;
    case 21: go<2, 1>(a, stream); break;
    case 22: go<2, 2>(a, stream); break;
    case 24: go<2, 4>(a, stream); break;
    case 31: go<3, 1>(a, stream); break;
    case 32: go<3, 2>(a, stream); break;
    default: go<3, 4>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace svdq
