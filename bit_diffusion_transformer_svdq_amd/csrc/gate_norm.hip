// The norms around a transformer block, fused with the block's gate and the
// residual scale, and the 8-bit token quantizer (gfx950).
//
//   u = post(y) * w_post            (post: none, RMS or layer norm, per row)
//   h = alpha x + gate * u
//   z = norm(h) * w * (1 + scale) + shift
//
// in fp32 from the unrounded h; h is rounded once to the residual stream's type,
// z once to bf16, or z goes straight to 8-bit codes: integers with one scale per row, or
// e4m3 with one per row and 128 channels, as the 8-bit linears read them.
// Adaptive-normalization blocks of a diffusion
// transformer take gate, scale and shift from the modulation projections
// (mind-verse.de, "Effiziente Optimierung von Diffusionsmodellen durch Nunchaku
// 4-Bit-Quantisierung", section "Nunchaku Lite: Nahtlose Integration in
// Diffusers", modulation layers).
//
// Bound by HBM: every element of x and y is read once and of h and z written
// once.  A row stays in registers between its reductions (mean, then centered
// squares: no cancellation), W waves per row and V vectors of 8 channels per lane;
// only rows of more than 16384 channels (16 waves of 3 or 4 vectors: 32 to 197 registers
// per lane go to scratch memory) do not fit: bf16 with both norms 1024 x 16384 31 us, 4.3
// TB/s, 1024 x 24576 79 us, 2.6 TB/s, 1024 x 32768 202 us, 1.3 TB/s.
// One row per workgroup (with W = 1: per wave) measured fastest: runs of rows with
// the shared vectors in registers and the next row in flight lost more to
// occupancy than they saved (4608 x 3072, with the loads in an earlier order: 23.6 to
// 26 us against 22.7).  Only with a smoothing vector, whose reciprocals are the
// dearest part, a workgroup takes a run of rows and keeps the reciprocals (quantizer
// 4608 x 3072: 16.2 -> 10.9 us).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8.h"

namespace svdq {
namespace {

// what z leaves as
enum NormOut { kOutBf16, kOutInt8, kOutFp8 };

constexpr int kWgWaves1 = 4;  // rows (waves) per workgroup when one wave owns a row

template <int W>
constexpr int threads_of() { return W == 1 ? 64 * kWgWaves1 : 64 * W; }

// the first row of this workgroup's (W == 1: wave's) run of `run` rows
template <int W>
__device__ __forceinline__ int first_row(int run) {
  const int owner = W == 1 ? (int)blockIdx.x * kWgWaves1 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)
                           : (int)blockIdx.x;
  return owner * run;  // below 2^25
}

__device__ __forceinline__ uint4 load8(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void load_f8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// 8 elements of the residual stream, as loaded
template <bool F32>
struct Stream8 {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void* x, size_t at) {
    if constexpr (F32) {
      const float* p = static_cast<const float*>(x) + at;
      lo = *reinterpret_cast<const uint4*>(p);
      hi = *reinterpret_cast<const uint4*>(p + 4);
    } else {
      lo = load8(static_cast<const uint16_t*>(x) + at);
    }
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    if constexpr (F32) {
      f[0] = __builtin_bit_cast(float, lo.x), f[1] = __builtin_bit_cast(float, lo.y);
      f[2] = __builtin_bit_cast(float, lo.z), f[3] = __builtin_bit_cast(float, lo.w);
      f[4] = __builtin_bit_cast(float, hi.x), f[5] = __builtin_bit_cast(float, hi.y);
      f[6] = __builtin_bit_cast(float, hi.z), f[7] = __builtin_bit_cast(float, hi.w);
    } else {
      unpack8(lo, f);
    }
  }
};

template <int W, int V, bool F32, NormOut kOut>
__global__ __launch_bounds__(threads_of<W>()) void gate_norm_kernel(const GateNormArgs a) {
  __shared__ float red_all[W > 1 ? 10 * W : 1];  // two sets of reduction slots, rows take turns
  const int row0 = first_row<W>(a.run), row_end = min(row0 + a.run, a.M);
  if (row0 >= row_end) return;
  const int lane0 = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int C8 = a.C >> 3;
  const float inv_c = 1.0f / (float)a.C;
  const bool has_y = a.y != nullptr, has_z = a.norm != kNormNone;

  // vector v of a lane: channels 8 i .. 8 i + 7, i = v * 64 W + lane; only the
  // last vector can lie past the row, its loads then repeat the last one
  int off[V];
#pragma unroll
  for (int v = 0; v < V; ++v) off[v] = 8 * min(v * 64 * W + lane0, C8 - 1);
  const bool live = (V - 1) * 64 * W + lane0 < C8;

  // the reciprocals stay in registers over a run, except where a row alone
  // fills them (16 waves, more than 8192 channels).  With one vector per lane (few
  // rows) they are taken behind the first row's loads (64 x 3072 5.1 -> 4.6 us),
  // with more ahead of the rows (4608 x 3072 25.7 -> 25.0 us)
  constexpr bool kKeep = kOut != kOutBf16 && (W < 16 || V == 1);
  float mu[kKeep ? V : 1][8];
  if constexpr (kKeep) {
    if (a.smooth != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        load_f8(a.smooth + off[v], mu[v]);
        if constexpr (V > 1) recip8(mu[v]);
      }
    }
  }
  auto load_all = [&](uint4 (&r)[V], const uint16_t* p, size_t at) {
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = load8(p + at + off[v]);
  };

  for (int row = row0; row < row_end; ++row) {
    float* red = red_all + (W > 1 ? 5 * W * (row & 1) : 0);
    // everything the first half of the row needs is requested at once, and the
    // vectors of the second half before its reductions: their round trips pass
    // side by side (against loads where they are used, 4608 x 3072 24.7 -> 20.7 us,
    // 8346 x 2304 fp32 with both norms 54.1 -> 47.3)
    Stream8<F32> px[V];
    uint4 py[V], pw[V], pg[V], ps[V];
    const size_t xo = (size_t)row * a.x_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) px[v].load(a.x, xo + off[v]);
    if (has_y) {
      load_all(py, a.y, (size_t)row * a.y_stride);
      if (a.gate != nullptr) load_all(pg, a.gate, (size_t)(row / a.gate_every) * a.gate_stride);
      if (a.post_weight != nullptr) load_all(pw, a.post_weight, 0);
    }
    float h[V][8], u[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      px[v].unpack(h[v]);
      if (has_y) unpack8(py[v], u[v]);
    }

    if (has_y) {
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
          if (a.post_weight != nullptr) {
            float w[8];
            unpack8(pw[v], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[v][e] *= r * w[e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[v][e] *= r;
          }
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.gate != nullptr) {
          float g[8];
          unpack8(pg[v], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] = __builtin_fmaf(g[e], u[v][e], a.alpha * h[v][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] = __builtin_fmaf(a.alpha, h[v][e], u[v][e]);
        }
      }
      const size_t ho = (size_t)row * a.h_stride;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < V - 1 || live) {
          if constexpr (F32) {
            float* p = static_cast<float*>(a.h) + ho + off[v];
            *reinterpret_cast<float4*>(p) = float4{h[v][0], h[v][1], h[v][2], h[v][3]};
            *reinterpret_cast<float4*>(p + 4) = float4{h[v][4], h[v][5], h[v][6], h[v][7]};
          } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + ho + off[v]) = pack8(h[v]);
          }
        }
    }
    if (!has_z) continue;

    const size_t mod = (size_t)(row / a.mod_every) * a.mod_stride;
    if (a.weight != nullptr) load_all(pw, a.weight, 0);
    if (a.scale != nullptr) load_all(pg, a.scale, mod);
    if (a.shift != nullptr) load_all(ps, a.shift, mod);
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
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] *= r;
      float w[8];
      if (a.weight != nullptr) {
        unpack8(pw[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= w[e];
      }
      if (a.scale != nullptr) {
        unpack8(pg[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = __builtin_fmaf(h[v][e], w[e], h[v][e]);
      }
      if (a.shift != nullptr) {
        unpack8(ps[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] += w[e];
      }
    }
    const size_t zo = (size_t)row * a.C;
    if constexpr (kOut == kOutBf16) {
      uint16_t* z = static_cast<uint16_t*>(a.z) + zo;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < V - 1 || live) *reinterpret_cast<uint4*>(z + off[v]) = pack8(h[v]);
    } else {
      float amax = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.smooth != nullptr) {
          float m[8];
          if constexpr (kKeep) {
            if (V == 1 && row == row0) recip8(mu[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = mu[v][e];
          } else {
            load_f8(a.smooth + off[v], m);
            recip8(m);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] *= m[e];
        }
        if constexpr (kOut == kOutFp8) amax = 0.f;  // of the lane's block of 128 channels, 16 lanes of one vector
        // (a lane past the row may hold what an update in place has already
        // written there: it takes no part)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          amax = (v < V - 1 || live) ? BitMaxOp::run(amax, __builtin_fabsf(h[v][e])) : amax;
        if constexpr (kOut == kOutFp8) {
          float s, inv;
          block_scale(max16(amax), s, inv);
          row_v2u c = {fp8_codes4(&h[v][0], inv), fp8_codes4(&h[v][4], inv)};
          if (inv == 0.f) c = row_v2u{0u, 0u};
          if (v < V - 1 || live) {
            *reinterpret_cast<row_v2u*>(static_cast<uint8_t*>(a.z) + zo + off[v]) = c;
            if ((lane0 & 15) == 0) a.scales[(size_t)(off[v] / kFp8Block) * a.M + row] = s;
          }
        }
      }
      if constexpr (kOut == kOutFp8) continue;
      amax = row_reduce<BitMaxOp, W>(amax, red, 4);
      float s, inv;
      token_scale(amax, s, inv);
      if (lane0 == 0) a.scales[row] = s;
      int8_t* q = static_cast<int8_t*>(a.z) + zo;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < V - 1 || live) {
          row_v2u c = {codes4(&h[v][0], inv), codes4(&h[v][4], inv)};
          if (inv == 0.f) c = row_v2u{0u, 0u};
          *reinterpret_cast<row_v2u*>(q + off[v]) = c;
        }
    }
  }
}

// x_hat = x, or bf16(fl32(x fl32(1/smooth))); s = fl32(max|x_hat| / 127);
// q = rint(x_hat fl32(1/s)).  The row is kept as packed bf16.
template <int W, int V, bool kSmooth>
__global__ __launch_bounds__(threads_of<W>()) void quant_int8_kernel(const QuantInt8Args a) {
  constexpr bool kKeep = V <= 3;  // reciprocals stay in registers over the run of rows
  __shared__ float red_all[W > 1 ? 2 * W : 1];
  const int row0 = first_row<W>(a.run), row_end = min(row0 + a.run, a.M);
  if (row0 >= row_end) return;
  const int lane0 = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int K8 = a.K >> 3;
  int off[V];
#pragma unroll
  for (int v = 0; v < V; ++v) off[v] = 8 * min(v * 64 * W + lane0, K8 - 1);
  const bool live = (V - 1) * 64 * W + lane0 < K8;
  float mu[kKeep ? V : 1][8];
  if constexpr (kSmooth && kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      load_f8(a.smooth + off[v], mu[v]);
      if constexpr (V > 1) recip8(mu[v]);  // (V == 1: as in the norm)
    }
  }
  for (int row = row0; row < row_end; ++row) {
    uint4 p[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = load8(a.x + (size_t)row * a.K + off[v]);
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      unpack8(p[v], f);
      if constexpr (kSmooth) {
        float m[8];
        if constexpr (kKeep) {
          if (V == 1 && row == row0) recip8(mu[v]);
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = mu[v][e];
        } else {
          load_f8(a.smooth + off[v], m);
          recip8(m);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= m[e];
        p[v] = pack8(f);
        unpack8(p[v], f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = BitMaxOp::run(amax, __builtin_fabsf(f[e]));
    }
    amax = row_reduce<BitMaxOp, W>(amax, red_all + (W > 1 ? W * (row & 1) : 0), 0);
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
}

template <int W>
dim3 grid_of(int M, int run) {
  const int owners = (M + run - 1) / run;
  return dim3(W == 1 ? (owners + kWgWaves1 - 1) / kWgWaves1 : owners);
}

template <int W, int V, NormOut kOut>
void gate_norm_go(const GateNormArgs& a, hipStream_t stream) {
  const dim3 grid = grid_of<W>(a.M, a.run), block(threads_of<W>());
  if (a.x_fp32) hipLaunchKernelGGL((gate_norm_kernel<W, V, true, kOut>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((gate_norm_kernel<W, V, false, kOut>), grid, block, 0, stream, a);
}
template <int W, int V>
void norm_bf16(const GateNormArgs& a, hipStream_t stream) { gate_norm_go<W, V, kOutBf16>(a, stream); }
template <int W, int V>
void norm_int8(const GateNormArgs& a, hipStream_t stream) { gate_norm_go<W, V, kOutInt8>(a, stream); }
template <int W, int V>
void norm_fp8(const GateNormArgs& a, hipStream_t stream) { gate_norm_go<W, V, kOutFp8>(a, stream); }

template <int W, int V, bool kSmooth>
void quant_go(const QuantInt8Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((quant_int8_kernel<W, V, kSmooth>), grid_of<W>(a.M, a.run), dim3(threads_of<W>()), 0, stream, a);
}
template <int W, int V>
void quant_smooth(const QuantInt8Args& a, hipStream_t stream) { quant_go<W, V, true>(a, stream); }
template <int W, int V>
void quant_plain(const QuantInt8Args& a, hipStream_t stream) { quant_go<W, V, false>(a, stream); }

// Waves per row: the fewest that leave a lane at most `per_lane` vectors, up to 16.
// With no more rows than compute units a row's latency counts and a lane takes
// one vector.
int waves_for(int64_t M, int c8, int per_lane) {
  if (M <= current_cus()) per_lane = 1;
  int w = 1;
  while (w < 16 && c8 > 64 * per_lane * w) w *= 2;
  return w;
}
// Measured on MI355X (us, W waves and V vectors; the best of each marked *):
//  gate norm  4608 x 1536: W1V3 12.5*, W2V2 13.0, W4V1 13.1    4608 x 5120: W4V3 37.1*, W8V2 40.8
//             4608 x 3072: W2V3 20.9*, W4V2 21.7, W8V1 24.6    4608 x 4096: W2V4 31.0, W4V2 29.4*, W8V1 31.5
//             8346 x 2304 fp32: W2V3 43.9*, W4V2 47.8          2304 x 8192: W4V4 31.5, W8V2 29.7*
//  quantizer  1333 x 1920: W1V4 3.5*, W2V2 3.7;  1000 x 16384: W4V8 9.8*, W16V2 10.4
//             4608 x 3072: W1V6 8.6*, W2V3 8.6*, W4V2 9.2, W8V1 10.1;  smoothed: W1V6 16.0, W2V3 10.8*, W4V2 11.2
//             4608 x 12288: W4V6 29.0, W8V3 28.9*, W16V2 32.0;  smoothed: W4V6 49.4, W8V3 34.5*, W16V2 36.6
//             smoothed, 2048 x 6144: W4V3 10.8*, W8V2 11.5;  1024 x 4608: W4V3 7.0*, W8V2 7.9;
//             512 x 3072: W2V3 4.8, W4V2 4.4*
//  The norm with 8-bit output and reciprocals: 4608 x 3072 W2V3 27.3, W4V2 24.1*, W8V1 29.5.
//  Codes with a scale per 128 channels take what int8 codes do and 0.7 to 1.3 us for the scales, which leave
//  one by one (4608 x 3072 24.6 against 23.9 us, with reciprocals 28.7 against 27.4).
constexpr int kNormPerLane = 3, kNormInt8PerLane = 2, kQuantPerLane = 8, kQuantSmoothPerLane = 3;

// Rows per run: one, or with a smoothing vector as many as leave kWavesPerCu
// waves per compute unit; more where the launch would come near 2^32 threads, its
// limit (2^24 rows of 4 waves).  Up to that many rows a run is one row, whose
// reciprocals then serve it alone (quantizer 1333 x 1920: 3.2 us, smoothed 4.8).
constexpr int kWavesPerCu = 32;
int run_for(int64_t M, int w, bool smooth) {
  const int64_t owners = std::min<int64_t>(smooth ? (int64_t)current_cus() * kWavesPerCu / w : M, (1 << 25) / w);
  return (int)((M + owners - 1) / owners);
}

}  // namespace

#define SVDQ_AT(go, W, V) \
  case 16 * W + V: go<W, V>(a, stream); break;
#define SVDQ_TO2(go, W) SVDQ_AT(go, W, 1) SVDQ_AT(go, W, 2)
#define SVDQ_TO3(go, W) SVDQ_TO2(go, W) SVDQ_AT(go, W, 3)
#define SVDQ_5TO8(go, W) SVDQ_AT(go, W, 5) SVDQ_AT(go, W, 6) SVDQ_AT(go, W, 7) SVDQ_AT(go, W, 8)
#define SVDQ_TO8(go, W) SVDQ_TO3(go, W) SVDQ_AT(go, W, 4) SVDQ_5TO8(go, W)

hipError_t launch_gate_norm(const GateNormArgs& args, hipStream_t stream) {
  GateNormArgs a = args;
  const bool q8 = a.scales != nullptr;
  const int c8 = a.C >> 3, w = waves_for(a.M, c8, q8 ? kNormInt8PerLane : kNormPerLane);
  const int v = (c8 + 64 * w - 1) / (64 * w);
  a.run = run_for(a.M, w, a.smooth != nullptr);
  if (q8 && a.fp8) {
    switch (16 * w + v) {
      SVDQ_TO2(norm_fp8, 1)
      SVDQ_TO2(norm_fp8, 2)
      SVDQ_TO2(norm_fp8, 4)
      SVDQ_TO2(norm_fp8, 8)
      SVDQ_TO3(norm_fp8, 16)
      SVDQ_AT(norm_fp8, 16, 4)
      default: return hipErrorInvalidValue;
    }
  } else if (q8) {
    switch (16 * w + v) {
      SVDQ_TO2(norm_int8, 1)
      SVDQ_TO2(norm_int8, 2)
      SVDQ_TO2(norm_int8, 4)
      SVDQ_TO2(norm_int8, 8)
      SVDQ_TO3(norm_int8, 16)
      SVDQ_AT(norm_int8, 16, 4)
      default: return hipErrorInvalidValue;
    }
  } else {
    switch (16 * w + v) {
      SVDQ_TO3(norm_bf16, 1)
      SVDQ_TO3(norm_bf16, 2)
      SVDQ_TO3(norm_bf16, 4)
      SVDQ_TO3(norm_bf16, 8)
      SVDQ_TO3(norm_bf16, 16)
      SVDQ_AT(norm_bf16, 16, 4)
      default: return hipErrorInvalidValue;
    }
  }
  return hipGetLastError();
}

hipError_t launch_quant_int8(const QuantInt8Args& args, hipStream_t stream) {
  QuantInt8Args a = args;
  const bool smooth = a.smooth != nullptr;
  const int k8 = a.K >> 3, w = waves_for(a.M, k8, smooth ? kQuantSmoothPerLane : kQuantPerLane);
  const int v = (k8 + 64 * w - 1) / (64 * w);
  a.run = run_for(a.M, w, smooth);
  if (smooth) {
    switch (16 * w + v) {
      SVDQ_TO3(quant_smooth, 1)
      SVDQ_TO3(quant_smooth, 2)
      SVDQ_TO3(quant_smooth, 4)
      SVDQ_TO3(quant_smooth, 8)
      SVDQ_TO8(quant_smooth, 16)
      default: return hipErrorInvalidValue;
    }
  } else {
    switch (16 * w + v) {
      SVDQ_TO8(quant_plain, 1)
      SVDQ_AT(quant_plain, 2, 1)
      SVDQ_5TO8(quant_plain, 2)
      SVDQ_AT(quant_plain, 4, 1)
      SVDQ_5TO8(quant_plain, 4)
      SVDQ_AT(quant_plain, 8, 1)
      SVDQ_5TO8(quant_plain, 8)
      SVDQ_TO8(quant_plain, 16)
      default: return hipErrorInvalidValue;
    }
  }
  return hipGetLastError();
}
#undef SVDQ_AT
#undef SVDQ_TO2
#undef SVDQ_TO3
#undef SVDQ_5TO8
#undef SVDQ_TO8

}  // namespace svdq
