// The 8-bit linear for up to 16 tokens on gfx950: a weight stream.
//
// With few tokens the product is bound by reading the weights once (N K bytes).
// A workgroup owns 16 weight rows and its 8 waves divide K: each wave reads its
// part of the rows straight into registers (16 rows x 64 bytes per load
// instruction), the same part of the token rows from L2, and accumulates one
// v_mfma_i32_16x16x64_i8 tile.  The waves' int32 partial tiles are added in LDS.
//
// Two steps of 64 k are loaded together and the next two while they are computed:
// deeper rings measured slower (1 token, 3072 -> 12288: 9.6 us with 2 steps, 11.1 with
// 4), as did 16 and 4 waves.  9.6 us is 3.9 TB/s over the weights, launch included;
// 3072 -> 3072 takes 4.9 us, 12288 -> 3072 11 to 12 us.  More rows per workgroup only pay where
// the tile kernel is faster still.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "row_device.h"
#include "w8a8.h"

namespace svdq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

constexpr int kBatch = 2;  // k steps of 64 loaded together

__global__ __launch_bounds__(kThreads) void w8a8_skinny_kernel(const W8a8Args a) {
  __shared__ __attribute__((aligned(16))) v4i red[kWaves][64];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int P = a.K >> 6;
  const int p0 = (int)((long)wave * P / kWaves), p1 = (int)((long)(wave + 1) * P / kWaves);

  const int8_t* wr = a.w + (size_t)(n0 + l16) * a.K + 16 * lq;  // N % 64 == 0
  const int8_t* ar = a.act + (size_t)min(l16, a.M - 1) * a.K + 16 * lq;
  v4i acc = {0, 0, 0, 0};

  struct Batch {
    v4i w[kBatch], a[kBatch];
  };
  // steps past the wave's range repeat its last one (their products are not
  // added), so every load of a batch is unconditional
  auto fetch = [&](Batch& f, int p) {
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int off = 64 * min(p + s, p1 - 1);
      f.w[s] = *reinterpret_cast<const v4i*>(wr + off);
      f.a[s] = *reinterpret_cast<const v4i*>(ar + off);
    }
  };
  auto add = [&](const Batch& f, int p) {
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (p + s < p1) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[s], f.a[s], acc, 0, 0, 0);
  };
  if (p0 < p1) {  // K may have fewer steps than the workgroup waves
    Batch f0, f1;
    fetch(f0, p0);
    int p = p0;
    for (; p + 2 * kBatch < p1; p += 2 * kBatch) {
      fetch(f1, p + kBatch);
      add(f0, p);
      fetch(f0, p + 2 * kBatch);
      add(f1, p + kBatch);
    }
    if (p + kBatch < p1) {
      fetch(f1, p + kBatch);
      add(f0, p);
      add(f1, p + kBatch);
    } else {
      add(f0, p);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  const int m = l16, n = n0 + 4 * lq;  // the lane's token and first of four channels
  if (m >= a.M) return;
  v4i s = red[0][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += red[w][lane];
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
    for (int v = 0; v < 4; ++v) o[v] = gelu_exp2(o[v]);
  }
  *reinterpret_cast<uint2*>(a.y + (size_t)m * a.N + n) = uint2{pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3])};
}

}  // namespace

hipError_t launch_w8a8_skinny(const W8a8Args& a, hipStream_t stream) {
  if (a.M > 16) return hipErrorInvalidValue;
  hipLaunchKernelGGL(w8a8_skinny_kernel, dim3(a.N / 16), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace svdq
