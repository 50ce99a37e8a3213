// The norms around a transformer block, fused with the block's gate and the
// residual scale, and the 8-bit token quantizer (gfx950).
//
//   u = post(y) * w_post            (post: none, RMS or layer norm, per row)
//   h = alpha x + gate * u
//   z = norm(h) * w * (1 + scale) + shift
//
// in fp32 from the unrounded h; h is rounded once to the residual stream's type,
// z once to bf16, or z goes straight to 8-bit codes with one scale per row, as
// the 8-bit linear reads it.  Adaptive-normalization blocks of a diffusion
// transformer take gate, scale and shift from the modulation projections
// (mind-verse.de, "Effiziente Optimierung von Diffusionsmodellen durch Nunchaku
// 4-Bit-Quantisierung", section "Nunchaku Lite: Nahtlose Integration in
// Diffusers", modulation layers).
//
// Bound by HBM: every element of x and y is read once and of h and z written
// once.  A row stays in registers between its reductions (mean, then centered
// squares: no cancellation), W waves per row, V vectors of 8 channels per lane.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "row_device.h"

namespace svdq {
namespace {

constexpr int kWgWaves1 = 4;  // rows (waves) per workgroup when one wave owns a row

template <int W>
constexpr int threads_of() { return W == 1 ? 64 * kWgWaves1 : 64 * W; }

// the row this wave works on (uniform)
template <int W>
__device__ __forceinline__ int row_of() {
  return W == 1 ? (int)blockIdx.x * kWgWaves1 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : (int)blockIdx.x;
}

template <int W, int V, bool F32, bool Q8>
__global__ __launch_bounds__(threads_of<W>()) void gate_norm_kernel(const GateNormArgs a) {
  __shared__ float red[W > 1 ? 5 * W : 1];
  const int row = row_of<W>();
  if (row >= a.M) return;  // W == 1 only: no barrier follows
  const int lane0 = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int C8 = a.C >> 3;
  const float inv_c = 1.0f / (float)a.C;

  // vector v of a lane: channels 8 i .. 8 i + 7, i = v * 64 W + lane; only the
  // last vector can lie past the row, its loads then repeat the last one
  int off[V];
#pragma unroll
  for (int v = 0; v < V; ++v) off[v] = 8 * min(v * 64 * W + lane0, C8 - 1);
  const bool live = (V - 1) * 64 * W + lane0 < C8;

  float h[V][8];
  if constexpr (F32) {
    const float* x = static_cast<const float*>(a.x) + (size_t)row * a.x_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float4 p = *reinterpret_cast<const float4*>(x + off[v]);
      const float4 q = *reinterpret_cast<const float4*>(x + off[v] + 4);
      h[v][0] = p.x, h[v][1] = p.y, h[v][2] = p.z, h[v][3] = p.w;
      h[v][4] = q.x, h[v][5] = q.y, h[v][6] = q.z, h[v][7] = q.w;
    }
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (size_t)row * a.x_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) unpack8(*reinterpret_cast<const uint4*>(x + off[v]), h[v]);
  }

  if (a.y != nullptr) {
    const uint16_t* y = a.y + (size_t)row * a.y_stride;
    float u[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) unpack8(*reinterpret_cast<const uint4*>(y + off[v]), u[v]);
    if (a.post != kNormNone) {
      float mean = 0.f;
      if (a.post == kNormLayer) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) s += (v < V - 1 || live) ? u[v][e] : 0.f;
        mean = row_reduce<SumOp, W>(s, red, 0) * inv_c;
      }
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[v][e] -= mean;
          ss = (v < V - 1 || live) ? __builtin_fmaf(u[v][e], u[v][e], ss) : ss;
        }
      const float r = 1.0f / sqrtf(__builtin_fmaf(row_reduce<SumOp, W>(ss, red, 1), inv_c, a.eps));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float w[8];
        if (a.post_weight != nullptr) {
          unpack8(*reinterpret_cast<const uint4*>(a.post_weight + off[v]), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[v][e] *= r * w[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[v][e] *= r;
        }
      }
    }
    const uint16_t* gate = a.gate + (size_t)(row / a.gate_every) * a.gate_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (a.gate != nullptr) {
        float g[8];
        unpack8(*reinterpret_cast<const uint4*>(gate + off[v]), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = __builtin_fmaf(g[e], u[v][e], a.alpha * h[v][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = __builtin_fmaf(a.alpha, h[v][e], u[v][e]);
      }
    }
    if constexpr (F32) {
      float* ho = static_cast<float*>(a.h) + (size_t)row * a.h_stride;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < V - 1 || live) {
          *reinterpret_cast<float4*>(ho + off[v]) = float4{h[v][0], h[v][1], h[v][2], h[v][3]};
          *reinterpret_cast<float4*>(ho + off[v] + 4) = float4{h[v][4], h[v][5], h[v][6], h[v][7]};
        }
    } else {
      uint16_t* ho = static_cast<uint16_t*>(a.h) + (size_t)row * a.h_stride;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < V - 1 || live) *reinterpret_cast<uint4*>(ho + off[v]) = pack8(h[v]);
    }
  }
  if (a.norm == kNormNone) return;

  float mean = 0.f;
  if (a.norm == kNormLayer) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (v < V - 1 || live) ? h[v][e] : 0.f;
    mean = row_reduce<SumOp, W>(s, red, 2) * inv_c;
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[v][e] -= mean;
      ss = (v < V - 1 || live) ? __builtin_fmaf(h[v][e], h[v][e], ss) : ss;
    }
  const float r = 1.0f / sqrtf(__builtin_fmaf(row_reduce<SumOp, W>(ss, red, 3), inv_c, a.eps));
  const size_t mod = (size_t)(row / a.mod_every) * a.mod_stride;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[v][e] *= r;
    float w[8];
    if (a.weight != nullptr) {
      unpack8(*reinterpret_cast<const uint4*>(a.weight + off[v]), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] *= w[e];
    }
    if (a.scale != nullptr) {
      unpack8(*reinterpret_cast<const uint4*>(a.scale + mod + off[v]), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = __builtin_fmaf(h[v][e], w[e], h[v][e]);
    }
    if (a.shift != nullptr) {
      unpack8(*reinterpret_cast<const uint4*>(a.shift + mod + off[v]), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] += w[e];
    }
  }
  if constexpr (!Q8) {
    uint16_t* z = static_cast<uint16_t*>(a.z) + (size_t)row * a.C;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < V - 1 || live) *reinterpret_cast<uint4*>(z + off[v]) = pack8(h[v]);
  } else {
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (a.smooth != nullptr) {
        float sm[8], mu[8];
        const float4 p = *reinterpret_cast<const float4*>(a.smooth + off[v]);
        const float4 q = *reinterpret_cast<const float4*>(a.smooth + off[v] + 4);
        sm[0] = p.x, sm[1] = p.y, sm[2] = p.z, sm[3] = p.w, sm[4] = q.x, sm[5] = q.y, sm[6] = q.z, sm[7] = q.w;
        recip8(sm, mu);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= mu[e];
      }
      // (a lane past the row may hold what an update in place has already
      // written there: it takes no part)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        amax = (v < V - 1 || live) ? BitMaxOp::run(amax, __builtin_fabsf(h[v][e])) : amax;
    }
    amax = row_reduce<BitMaxOp, W>(amax, red, 4);
    float s, inv;
    token_scale(amax, s, inv);
    if (lane0 == 0) a.scales[row] = s;
    int8_t* q = static_cast<int8_t*>(a.z) + (size_t)row * a.C;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < V - 1 || live) {
        row_v2u c = {codes4(&h[v][0], inv), codes4(&h[v][4], inv)};
        if (inv == 0.f) c = row_v2u{0u, 0u};
        *reinterpret_cast<row_v2u*>(q + off[v]) = c;
      }
  }
}

// x_hat = x, or bf16(fl32(x fl32(1/smooth))); s = fl32(max|x_hat| / 127);
// q = rint(x_hat fl32(1/s)).  The row is kept as packed bf16.
template <int W, int V, bool kSmooth>
__global__ __launch_bounds__(threads_of<W>()) void quant_int8_kernel(const QuantInt8Args a) {
  __shared__ float red[W > 1 ? W : 1];
  const int row = row_of<W>();
  if (row >= a.M) return;  // W == 1 only
  const int lane0 = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int K8 = a.K >> 3;
  int off[V];
#pragma unroll
  for (int v = 0; v < V; ++v) off[v] = 8 * min(v * 64 * W + lane0, K8 - 1);
  const bool live = (V - 1) * 64 * W + lane0 < K8;
  const uint16_t* x = a.x + (size_t)row * a.K;
  uint4 p[V];
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = *reinterpret_cast<const uint4*>(x + off[v]);
  float amax = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f[8];
    unpack8(p[v], f);
    if constexpr (kSmooth) {
      float sm[8], mu[8];
      const float4 s0 = *reinterpret_cast<const float4*>(a.smooth + off[v]);
      const float4 s1 = *reinterpret_cast<const float4*>(a.smooth + off[v] + 4);
      sm[0] = s0.x, sm[1] = s0.y, sm[2] = s0.z, sm[3] = s0.w, sm[4] = s1.x, sm[5] = s1.y, sm[6] = s1.z, sm[7] = s1.w;
      recip8(sm, mu);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= mu[e];
      p[v] = pack8(f);
      unpack8(p[v], f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = BitMaxOp::run(amax, __builtin_fabsf(f[e]));
  }
  amax = row_reduce<BitMaxOp, W>(amax, red, 0);
  float s, inv;
  token_scale(amax, s, inv);
  if (lane0 == 0) a.scales[row] = s;
  int8_t* q = a.codes + (size_t)row * a.K;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f[8];
    unpack8(p[v], f);
    row_v2u c = {codes4(&f[0], inv), codes4(&f[4], inv)};
    if (inv == 0.f) c = row_v2u{0u, 0u};
    if (v < V - 1 || live) *reinterpret_cast<row_v2u*>(q + off[v]) = c;
  }
}

template <int W, int V>
void gate_norm_go(const GateNormArgs& a, hipStream_t stream) {
  const dim3 grid(W == 1 ? (a.M + kWgWaves1 - 1) / kWgWaves1 : a.M), block(threads_of<W>());
  if (a.x_fp32) {
    if (a.scales) hipLaunchKernelGGL((gate_norm_kernel<W, V, true, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((gate_norm_kernel<W, V, true, false>), grid, block, 0, stream, a);
  } else {
    if (a.scales) hipLaunchKernelGGL((gate_norm_kernel<W, V, false, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((gate_norm_kernel<W, V, false, false>), grid, block, 0, stream, a);
  }
}

template <int W, int V>
void quant_go(const QuantInt8Args& a, hipStream_t stream) {
  const dim3 grid(W == 1 ? (a.M + kWgWaves1 - 1) / kWgWaves1 : a.M), block(threads_of<W>());
  if (a.smooth) hipLaunchKernelGGL((quant_int8_kernel<W, V, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((quant_int8_kernel<W, V, false>), grid, block, 0, stream, a);
}

// waves per row: one while the row fits its registers and there are rows
// enough to occupy every SIMD, else as many as keep the row in registers
int waves_for(int64_t M, int c8) {
  if (c8 <= 512 && M >= 2 * 4 * (int64_t)current_cus()) return 1;
  if (c8 <= 1024) return 4;
  return c8 <= 2048 ? 8 : 16;
}

}  // namespace

hipError_t launch_gate_norm(const GateNormArgs& a, hipStream_t stream) {
  const int c8 = a.C >> 3;
  const int w = waves_for(a.M, c8);
  const int v = (c8 + 64 * w - 1) / (64 * w);
#define SVDQ_CASE(W, V) \
  case 16 * W + V: gate_norm_go<W, V>(a, stream); break;
  switch (16 * w + v) {
    SVDQ_CASE(1, 1) SVDQ_CASE(1, 2) SVDQ_CASE(1, 3) SVDQ_CASE(1, 4)
    SVDQ_CASE(1, 5) SVDQ_CASE(1, 6) SVDQ_CASE(1, 7) SVDQ_CASE(1, 8)
    SVDQ_CASE(4, 1) SVDQ_CASE(4, 2) SVDQ_CASE(4, 3) SVDQ_CASE(4, 4)
    SVDQ_CASE(8, 3) SVDQ_CASE(8, 4) SVDQ_CASE(16, 3) SVDQ_CASE(16, 4)
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_quant_int8(const QuantInt8Args& a, hipStream_t stream) {
  const int k8 = a.K >> 3;
  const int w = k8 > 2048 ? 16 : k8 > 1024 ? 4 : waves_for(a.M, k8);
  const int v = (k8 + 64 * w - 1) / (64 * w);
#undef SVDQ_CASE
#define SVDQ_CASE(W, V) \
  case 16 * W + V: quant_go<W, V>(a, stream); break;
  switch (16 * w + v) {
    SVDQ_CASE(1, 1) SVDQ_CASE(1, 2) SVDQ_CASE(1, 3) SVDQ_CASE(1, 4)
    SVDQ_CASE(1, 5) SVDQ_CASE(1, 6) SVDQ_CASE(1, 7) SVDQ_CASE(1, 8)
    SVDQ_CASE(4, 1) SVDQ_CASE(4, 2) SVDQ_CASE(4, 3) SVDQ_CASE(4, 4)
    SVDQ_CASE(4, 5) SVDQ_CASE(4, 6) SVDQ_CASE(4, 7) SVDQ_CASE(4, 8)
    SVDQ_CASE(16, 3) SVDQ_CASE(16, 4) SVDQ_CASE(16, 5) SVDQ_CASE(16, 6) SVDQ_CASE(16, 7) SVDQ_CASE(16, 8)
    default: return hipErrorInvalidValue;
  }
#undef SVDQ_CASE
  return hipGetLastError();
}

}  // namespace svdq
