// Rotary positions with several axes (time, height, width, ...) on gfx950:
// tables of cosines and sines, and the turn of Q and K heads with an optional
// RMSNorm per head before it.
//
// A token has one position per axis; the rotary width R is divided among the
// axes, and angle i (i < R/2) of a token is its position on the axis that owns
// i times a rate that falls geometrically, over the axis's own width or over
// all of R (RoFormer, Su et al., 2021, for one axis).  The fused QKV operator of
// the W4A4 linear takes such tables (mind-verse.de, "Effiziente Optimierung von
// Diffusionsmodellen durch Nunchaku 4-Bit-Quantisierung", section
// "Quantisierung von Modellen mit strukturellen Umschreibungen"); the kernel
// here turns the Q and K of any other projection.
//
// Angles: the rates arrive in revolutions per unit of position, as doubles;
// the product with the position and its reduction to [-1/2, 1/2] are done in
// double (three operations per angle), so a far position keeps the 2^-24 of a
// near one, and sincospif needs no reduction of its own.
//
// The turn is bound by HBM: Q and K are read and written once.  A workgroup
// computes the angles of its tokens once, in LDS, and a lane keeps its chunk's
// cosines and sines in registers for all heads of a token.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "row_device.h"

namespace svdq {
namespace {

constexpr int kThreads = 256;

struct Rates {
  double per_unit[kRopeMaxAngles];  // revolutions per unit of position
  uint8_t axis[kRopeMaxAngles];
};

struct TurnArgs {
  RopeArgs a;
  Rates f;
  int tokens;  // per workgroup
  int heads_per_wg;
};

struct TableArgs {
  const void* positions;
  float* cos;
  float* sin;
  Rates f;
  int n_axes, half, pos_int;
  int M;
};

__device__ __forceinline__ float2 angle_of(const void* positions, int pos_int, int64_t at, double rate) {
  const double p = pos_int ? (double)static_cast<const int32_t*>(positions)[at]
                           : (double)static_cast<const float*>(positions)[at];
  const double rev = p * rate;
  const float r = (float)(rev - __builtin_rint(rev));
  float s, c;
  sincospif(2.0f * r, &s, &c);
  return float2{c, s};
}

__global__ __launch_bounds__(kThreads) void rope_tables_kernel(const TableArgs a) {
  const int64_t n = (int64_t)a.M * a.half;
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (at >= n) return;
  const int64_t m = at / a.half;
  const int i = (int)(at - m * a.half);
  const float2 cs = angle_of(a.positions, a.pos_int, m * a.n_axes + a.f.axis[i], a.f.per_unit[i]);
  a.cos[at] = cs.x;
  a.sin[at] = cs.y;
}

template <int VEC>
struct Chunk;
template <>
struct Chunk<8> {
  typedef uint4 T;
  static __device__ __forceinline__ void unpack(const uint4& p, float (&f)[8]) { unpack8(p, f); }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) { return pack8(f); }
};
template <>
struct Chunk<4> {
  typedef uint2 T;
  static __device__ __forceinline__ void unpack(const uint2& p, float (&f)[4]) {
    f[0] = bf16_lo(p.x), f[1] = bf16_hi(p.x), f[2] = bf16_lo(p.y), f[3] = bf16_hi(p.y);
  }
  static __device__ __forceinline__ uint2 pack(const float (&f)[4]) {
    return uint2{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3])};
  }
};

// the sum over the aligned group of `lanes` (a power of two) that holds a head
__device__ __forceinline__ float group_sum(float x, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor(x, o);
  return x;
}

// VEC channels per lane; a head takes `lanes` = the power of two >= D / VEC
// lanes, those past D / VEC idle.
template <int VEC, bool kHalves, bool kNorm>
__global__ __launch_bounds__(kThreads) void rope_turn_kernel(const TurnArgs t) {
  typedef typename Chunk<VEC>::T Pack;
  constexpr int kPer = 4;  // heads whose loads are in flight together
  extern __shared__ __align__(16) float2 ang[];
  const RopeArgs& a = t.a;
  const int half = a.half;
  const int tid = threadIdx.x;
  const int64_t m0 = (int64_t)blockIdx.x * t.tokens;
  const int nt = (int)min((int64_t)t.tokens, (int64_t)a.M - m0);
  for (int e = tid; e < nt * half; e += kThreads) {
    const int tok = e / half, i = e - tok * half;
    const int64_t p = (m0 + tok) % a.pos_rows;
    ang[e] = angle_of(a.positions, a.pos_int, p * a.n_axes + t.f.axis[i], t.f.per_unit[i]);
  }
  __syncthreads();

  const int lanes = a.lanes;                 // per head
  const int sub = tid & (lanes - 1);         // chunk of the head
  const int ch = sub * VEC;
  const bool live = ch < a.D;
  const int chc = live ? ch : 0;             // idle lanes repeat chunk 0 (never stored)
  const bool turned = ch < 2 * half;
  const int groups = kThreads / lanes;
  const int heads = a.q_heads + a.k_heads;
  const int h_end = min(heads, (int)(blockIdx.y + 1) * t.heads_per_wg);
  // halves: channel i turns with channel i + half, which is `shift` lanes away
  const bool first = ch < half;
  const int shift = half / VEC;
  const int mate = kHalves ? (turned ? (first ? sub + shift : sub - shift) : sub) : sub;
  const int mate_lane = ((tid & 63) & ~(lanes - 1)) | mate;

  float wq[VEC], wk[VEC], wq2[VEC], wk2[VEC];  // norm weights of the lane's channels and its mate's
  if constexpr (kNorm) {
    Chunk<VEC>::unpack(*reinterpret_cast<const Pack*>(a.q_norm + chc), wq);
    if (a.k_norm != nullptr) Chunk<VEC>::unpack(*reinterpret_cast<const Pack*>(a.k_norm + chc), wk);
    if constexpr (kHalves) {
      const int c2 = live ? mate * VEC : 0;
      Chunk<VEC>::unpack(*reinterpret_cast<const Pack*>(a.q_norm + c2), wq2);
      if (a.k_norm != nullptr) Chunk<VEC>::unpack(*reinterpret_cast<const Pack*>(a.k_norm + c2), wk2);
    }
  }
  const float inv_d = 1.0f / (float)a.D;

  for (int tok = 0; tok < nt; ++tok) {
    const int64_t m = m0 + tok;
    float c[VEC], s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = kHalves ? (first ? ch : ch - half) + e : (ch + e) >> 1;
      const bool te = ch + e < 2 * half;  // R need not end with a chunk
      const float2 cs = ang[tok * half + (te ? i : 0)];
      c[e] = te ? cs.x : 1.f;
      s[e] = te ? cs.y : 0.f;
      if (kHalves ? first : (e & 1) == 0) s[e] = -s[e];
    }
    for (int h0 = (int)blockIdx.y * t.heads_per_wg + tid / lanes; h0 < h_end; h0 += kPer * groups) {
      Pack p[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int h = min(h0 + u * groups, h_end - 1);
        const uint16_t* src = h < a.q_heads ? a.q + m * a.q_stride + (int64_t)h * a.D
                                            : a.k + m * a.k_stride + (int64_t)(h - a.q_heads) * a.D;
        p[u] = *reinterpret_cast<const Pack*>(src + chc);
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int h = h0 + u * groups;
        const bool is_q = h < a.q_heads;
        float v[VEC], o[VEC], w[VEC];
        Chunk<VEC>::unpack(p[u], v);
        if constexpr (kHalves) {
          Pack b;
          uint32_t* dst = reinterpret_cast<uint32_t*>(&b);
          const uint32_t* from = reinterpret_cast<const uint32_t*>(&p[u]);
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) dst[e] = (uint32_t)__shfl((int)from[e], mate_lane);
          Chunk<VEC>::unpack(b, w);
        }
        if constexpr (kNorm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
          ss = group_sum(live ? ss : 0.f, lanes);
          const float r = 1.0f / sqrtf(__builtin_fmaf(ss, inv_d, a.eps));
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            v[e] *= r * (is_q ? wq[e] : wk[e]);
            if constexpr (kHalves) w[e] *= r * (is_q ? wq2[e] : wk2[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float other = kHalves ? w[e] : v[e ^ 1];
          o[e] = __builtin_fmaf(v[e], c[e], other * s[e]);
        }
        if (live && h < h_end) {
          uint16_t* dst = is_q ? a.q_out + m * a.qo_stride + (int64_t)h * a.D
                               : a.k_out + m * a.ko_stride + (int64_t)(h - a.q_heads) * a.D;
          *reinterpret_cast<Pack*>(dst + ch) = Chunk<VEC>::pack(o);
        }
      }
    }
  }
}

// rate of angle i in revolutions: theta^(-2j/d) / (2 pi), j and d within the
// axis, or theta^(-2i/R) / (2 pi).  A running product in extended precision
// (error below 2^-56 over 128 steps).
void make_rates(const RopeAxes& x, Rates& f) {
  const long double turn = 6.283185307179586476925286766559L;
  const long double lt = std::log((long double)x.theta);
  int at = 0;
  long double all = 1.0L / turn;
  const long double all_step = std::exp(-lt / (long double)x.half);
  for (int ax = 0; ax < x.n; ++ax) {
    const int pairs = x.width[ax] / 2;
    const long double step = pairs > 0 ? std::exp(-lt / (long double)pairs) : 1.0L;
    long double v = 1.0L / turn;
    for (int j = 0; j < pairs; ++j, ++at) {
      f.per_unit[at] = (double)(x.shared ? all : v);
      f.axis[at] = (uint8_t)ax;
      v *= step;
      all *= all_step;
    }
  }
}

template <int VEC, bool kHalves, bool kNorm>
void turn_go(const TurnArgs& t, dim3 grid, size_t lds, hipStream_t stream) {
  hipLaunchKernelGGL((rope_turn_kernel<VEC, kHalves, kNorm>), grid, dim3(kThreads), lds, stream, t);
}

}  // namespace

hipError_t launch_rope_tables(const void* positions, bool pos_int, const RopeAxes& axes, int64_t M, float* cos,
                              float* sin, hipStream_t stream) {
  TableArgs a{};
  a.positions = positions;
  a.cos = cos;
  a.sin = sin;
  a.n_axes = axes.n;
  a.half = axes.half;
  a.pos_int = pos_int;
  a.M = (int)M;
  make_rates(axes, a.f);
  const int64_t n = M * axes.half;
  hipLaunchKernelGGL(rope_tables_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_rope_axes(const RopeArgs& args, const RopeAxes& axes, bool halves, hipStream_t stream) {
  TurnArgs t{};
  t.a = args;
  t.a.n_axes = axes.n;
  t.a.half = axes.half;
  make_rates(axes, t.f);
  // 16-byte chunks, except that halves need whole chunks up to R/2
  const int vec = halves && axes.half % 8 != 0 ? 4 : 8;
  int lanes = 1;
  while (lanes * vec < args.D) lanes *= 2;
  t.a.lanes = lanes;
  const int groups = kThreads / lanes;
  const int heads = args.q_heads + args.k_heads;
  // tokens per workgroup: as many as its threads have angles for, while the
  // launch still has four workgroups per compute unit; with fewer tokens than
  // that the heads are divided as well (each workgroup then computes the few
  // angles again)
  const int cus = current_cus();
  t.tokens = std::max(1, kThreads / std::max(1, axes.half));
  while (t.tokens > 1 && (int64_t)args.M < (int64_t)t.tokens * 4 * cus) t.tokens /= 2;
  const int gx = (int)((args.M + t.tokens - 1) / t.tokens);
  const int most = (heads + groups - 1) / groups;  // one head per lane group at least
  const int gy = std::max(1, std::min(most, (2 * cus) / std::max(1, gx)));
  t.heads_per_wg = (heads + gy - 1) / gy;
  t.heads_per_wg = (t.heads_per_wg + groups - 1) / groups * groups;
  const dim3 grid(gx, (heads + t.heads_per_wg - 1) / t.heads_per_wg);
  const size_t lds = (size_t)t.tokens * std::max(1, axes.half) * sizeof(float2);
  const bool norm = args.q_norm != nullptr;
  if (vec == 8) {
    if (halves) norm ? turn_go<8, true, true>(t, grid, lds, stream) : turn_go<8, true, false>(t, grid, lds, stream);
    else norm ? turn_go<8, false, true>(t, grid, lds, stream) : turn_go<8, false, false>(t, grid, lds, stream);
  } else {
    norm ? turn_go<4, true, true>(t, grid, lds, stream) : turn_go<4, true, false>(t, grid, lds, stream);
  }
  return hipGetLastError();
}

}  // namespace svdq
