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
// Angles: the rates arrive in quarter turns per unit of position, each as a double
// and what that leaves.  The product with the position, unrounded, its reduction to
// [-1/2, 1/2] quarter turns and the Taylor series of sine and cosine (to t^13 and t^14:
// below 2^-45 at pi/4) are done in double, about 22 operations per angle.  Up to |position| = 2^31 (any int32) the angle is then within
// 2^-28 for theta of 1e4 and more (one rate in 64 bits, below 2^-60 of it), and each value
// is rounded to fp32 once; with the double alone it is off by up to 2^-21.6 there.
//
// The turn is bound by HBM: Q and K are read and written once.  A workgroup
// computes the angles of its tokens once, in LDS, for all their heads, while the
// first of them are being loaded.  4608 tokens of 24 + 24 heads of 128: 22 us normed,
// 5.1 TB/s; 32760 tokens of 12 + 12: 72 us, 5.6 TB/s (a copy of 1 GiB runs at 5.2 TB/s).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "row_device.h"

namespace svdq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // per workgroup; with 8192 heads 2^15 items

// one 16-byte load per angle
struct Rate {
  double per_unit;  // quarter turns per unit of position
  float rest;       // what the double leaves of the rate
  int axis;
};
struct Rates {
  Rate of[kRopeMaxAngles];
};

struct TurnArgs {
  RopeArgs a;
  Rates f;
  int tokens;  // per workgroup
  int heads_per_wg;
  uint32_t heads_magic;  // ceil(2^32 / heads_per_wg)
};

struct TableArgs {
  const void* positions;
  float* cos;
  float* sin;
  Rates f;
  int n_axes, half, pos_int;
  int M;
};

// the row of positions starts at `row`
__device__ __forceinline__ float2 angle_of(const void* positions, int pos_int, int64_t row, const Rate& f) {
  const int64_t at = row + f.axis;
  const double rate = f.per_unit, rest = (double)f.rest;
  const double p = pos_int ? (double)static_cast<const int32_t*>(positions)[at]
                           : (double)static_cast<const float*>(positions)[at];
  const double turns = p * rate, quarter = __builtin_rint(turns);
  // the product again, unrounded, less its quarters.  Past 2^45 quarters (fp32 positions
  // 2^22 apart) what the rounding leaves would pass the series' range in the end: those
  // turn by whole quarters (NaN where they are not finite)
  double t = __builtin_fma(p, rest, __builtin_fma(p, rate, -quarter));
  if (!(__builtin_fabs(turns) < 0x1p45)) t = quarter * 0.0;
  t *= 1.5707963267948966;
  const double t2 = t * t;
  double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
  s = __builtin_fma(s, t2, -1.0 / 39916800.0);
  s = __builtin_fma(s, t2, 1.0 / 362880.0);
  s = __builtin_fma(s, t2, -1.0 / 5040.0);
  s = __builtin_fma(s, t2, 1.0 / 120.0);
  s = __builtin_fma(s, t2, -1.0 / 6.0);
  s = __builtin_fma(s * t2, t, t);
  c = __builtin_fma(c, t2, 1.0 / 479001600.0);
  c = __builtin_fma(c, t2, -1.0 / 3628800.0);
  c = __builtin_fma(c, t2, 1.0 / 40320.0);
  c = __builtin_fma(c, t2, -1.0 / 720.0);
  c = __builtin_fma(c, t2, 1.0 / 24.0);
  c = __builtin_fma(c, t2, -0.5);
  c = __builtin_fma(c, t2, 1.0);
  // the quarter within its turn, 0 to 3 (exact; for a position that is not finite
  // s and c are NaN whatever it is)
  const double k = quarter - 4.0 * __builtin_floor(quarter * 0.25);
  const bool odd = k == 1.0 || k == 3.0;
  const float fs = (float)s, fc = (float)c;
  const float x = odd ? fs : fc, y = odd ? fc : fs;
  return float2{k == 1.0 || k == 2.0 ? -x : x, k >= 2.0 ? -y : y};
}

__global__ __launch_bounds__(kThreads) void rope_tables_kernel(const TableArgs a) {
  const int64_t n = (int64_t)a.M * a.half;
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (at >= n) return;
  const int64_t m = at / a.half;
  const int i = (int)(at - m * a.half);
  const float2 cs = angle_of(a.positions, a.pos_int, m * a.n_axes, a.f.of[i]);
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
  if (lanes > 1) x += dpp_mov<0xB1>(x);    // quad_perm 1 0 3 2
  if (lanes > 2) x += dpp_mov<0x4E>(x);    // quad_perm 2 3 0 1
  if (lanes > 4) x += dpp_mov<0x141>(x);   // mirror of 8 lanes
  if (lanes > 8) x += dpp_mov<0x140>(x);   // mirror of 16 lanes
  if (lanes > 16) {
    const row_u32 u = __builtin_bit_cast(row_u32, x);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = __builtin_bit_cast(float, (row_u32)p[0]) + __builtin_bit_cast(float, (row_u32)p[1]);
  }
  if (lanes > 32) {
    const row_u32 u = __builtin_bit_cast(row_u32, x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = __builtin_bit_cast(float, (row_u32)p[0]) + __builtin_bit_cast(float, (row_u32)p[1]);
  }
  return x;
}

// 1 / sqrt(x) within 2 fp32 ulp; below the range of v_rsq_f32 the IEEE operations
__device__ __forceinline__ float rsqrt_of(float x) {
  float r = __builtin_amdgcn_rsqf(x);
  if (x < 0x1p-120f) r = 1.0f / sqrtf(x);
  return r;
}

// VEC channels per lane; a head takes `lanes` = the power of two >= D / VEC
// lanes, those past D / VEC idle (4608 tokens of 48 normed heads: D = 64 4.7 TB/s, 80
// 3.8, 96 4.5, 128 5.1, 256 4.4).  The (token, head) items of the workgroup are
// dealt to its lane groups in order, kPer items of a group in flight together.
template <int VEC, bool kHalves, bool kNorm>
__global__ __launch_bounds__(kThreads) void rope_turn_kernel(const TurnArgs t) {
  typedef typename Chunk<VEC>::T Pack;
  constexpr int kPer = 2;
  extern __shared__ __align__(16) float2 ang[];
  const RopeArgs& a = t.a;
  const int half = a.half;
  const int tid = threadIdx.x;
  const int64_t m0 = (int64_t)blockIdx.x * t.tokens;
  const int nt = (int)min((int64_t)t.tokens, (int64_t)a.M - m0);
  const int lanes = a.lanes;                 // per head
  const int sub = tid & (lanes - 1);         // chunk of the head
  const int ch = sub * VEC;
  const bool live = ch < a.D;
  const int chc = live ? ch : 0;             // idle lanes repeat chunk 0 (never stored)
  const bool turned = ch < 2 * half;
  const int groups = kThreads / lanes;
  const int head0 = (int)blockIdx.y * t.heads_per_wg;
  const int heads = min(t.heads_per_wg, a.q_heads + a.k_heads - head0);  // of this workgroup
  const int items = nt * heads;
  // halves: channel i turns with channel i + half, which is half / VEC lanes away
  const bool first = ch < half;
  const int mate = kHalves && turned ? (first ? sub + half / VEC : sub - half / VEC) : sub;
  const int mate_lane = ((tid & 63) & ~(lanes - 1)) | mate;
  const int angle0 = kHalves ? (first ? ch : ch - half) : ch >> 1;  // the chunk's first angle
  const float sign = first ? -1.f : 1.f;

  Pack wq{}, wk{}, wq2{}, wk2{};  // norm weights of the lane's channels and its mate's
  if constexpr (kNorm) {
    wq = *reinterpret_cast<const Pack*>(a.q_norm + chc);
    if (a.k_norm != nullptr) wk = *reinterpret_cast<const Pack*>(a.k_norm + chc);
    if constexpr (kHalves) {
      const int c2 = live ? mate * VEC : 0;
      wq2 = *reinterpret_cast<const Pack*>(a.q_norm + c2);
      if (a.k_norm != nullptr) wk2 = *reinterpret_cast<const Pack*>(a.k_norm + c2);
    }
  }
  const float inv_d = 1.0f / (float)a.D;

  struct Batch {
    Pack p[kPer];
    int tok[kPer], head[kPer];
  };
  auto load = [&](Batch& b, int it0) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int it = it0 + u * groups;
      if (it < items) {
        // items < 2^16, heads <= 2^13: the product with ceil(2^32 / heads) divides
        // exactly (one head has no such factor, the last part of divided heads another)
        b.tok[u] = heads == 1 ? it : heads == t.heads_per_wg ? (int)__umulhi((row_u32)it, t.heads_magic) : it / heads;
        b.head[u] = head0 + it - b.tok[u] * heads;
        const int64_t m = m0 + b.tok[u];
        const uint16_t* src = b.head[u] < a.q_heads ? a.q + m * a.q_stride + (int64_t)b.head[u] * a.D
                                                    : a.k + m * a.k_stride + (int64_t)(b.head[u] - a.q_heads) * a.D;
        b.p[u] = *reinterpret_cast<const Pack*>(src + chc);
      }
    }
  };
  auto turn = [&](const Batch& b, int it0) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (it0 + u * groups >= items) continue;  // uniform within a head's lanes
      const bool is_q = b.head[u] < a.q_heads;
      float v[VEC], o[VEC], w[VEC];
      Chunk<VEC>::unpack(b.p[u], v);
      if constexpr (kHalves) {
        Pack other;
        uint32_t* dst = reinterpret_cast<uint32_t*>(&other);
        const uint32_t* from = reinterpret_cast<const uint32_t*>(&b.p[u]);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) dst[e] = (uint32_t)__shfl((int)from[e], mate_lane);
        Chunk<VEC>::unpack(other, w);
      }
      if constexpr (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
        ss = group_sum(live ? ss : 0.f, lanes);
        const float r = rsqrt_of(__builtin_fmaf(ss, inv_d, a.eps));
        float g[VEC];
        Chunk<VEC>::unpack(is_q ? wq : wk, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] *= r * g[e];
        if constexpr (kHalves) {
          Chunk<VEC>::unpack(is_q ? wq2 : wk2, g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) w[e] *= r * g[e];
        }
      }
      if (turned) {
        const float2* cs = ang + b.tok[u] * half + angle0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if constexpr (kHalves) {
            o[e] = __builtin_fmaf(v[e], cs[e].x, sign * w[e] * cs[e].y);
          } else {
            // (R need not end with a chunk)
            const bool te = ch + e < 2 * half;
            const float2 x = cs[te ? e >> 1 : 0];
            const float y = (e & 1) == 0 ? -v[e ^ 1] * x.y : v[e ^ 1] * x.y;
            o[e] = te ? __builtin_fmaf(v[e], x.x, y) : v[e];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = v[e];
      }
      if (live) {
        const int64_t m = m0 + b.tok[u];
        uint16_t* dst = is_q ? a.q_out + m * a.qo_stride + (int64_t)b.head[u] * a.D
                             : a.k_out + m * a.ko_stride + (int64_t)(b.head[u] - a.q_heads) * a.D;
        // streaming (non-temporal) stores: nothing here reads them back (25.5 -> 22.7 us
        // on 4608 tokens of 48 heads of 128, normed)
        typedef row_u32 Words __attribute__((ext_vector_type(VEC / 2)));
        __builtin_nontemporal_store(__builtin_bit_cast(Words, Chunk<VEC>::pack(o)), reinterpret_cast<Words*>(dst + ch));
      }
    }
  };

  // the first items are on their way while the angles are computed, the next
  // ones while a batch is turned
  const int step = kPer * groups;
  int it = tid / lanes;
  Batch b0, b1;
  load(b0, it);
  for (int e = tid; e < nt * half; e += kThreads) {
    const int tok = e / half, i = e - tok * half;
    const int64_t p = (m0 + tok) % a.pos_rows;
    ang[e] = angle_of(a.positions, a.pos_int, p * a.n_axes, t.f.of[i]);
  }
  __syncthreads();
  for (; it < items; it += 2 * step) {
    load(b1, it + step);
    turn(b0, it);
    load(b0, it + 2 * step);
    turn(b1, it + step);
  }
}

// rate of angle i in quarter turns: theta^(-2j/d) / (pi/2), j and d within the
// axis, or theta^(-2i/R) / (pi/2).  A running product in extended precision
// (step j is off by about 1.5 j 2^-63 of the rate: below 2^-60 of the fastest one
// for theta of 1e4 and more, where the rate falls as j grows).
void make_rates(const RopeAxes& x, Rates& f) {
  const long double quarter = 1.5707963267948966192313216916398L;
  const long double lt = std::log((long double)x.theta);
  int at = 0;
  long double all = 1.0L / quarter;
  const long double all_step = std::exp(-lt / (long double)x.half);
  for (int ax = 0; ax < x.n; ++ax) {
    const int pairs = x.width[ax] / 2;
    const long double step = pairs > 0 ? std::exp(-lt / (long double)pairs) : 1.0L;
    long double v = 1.0L / quarter;
    for (int j = 0; j < pairs; ++j, ++at) {
      const long double rate = x.shared ? all : v;
      const double top = (double)rate;
      f.of[at] = Rate{top, (float)(rate - (long double)top), ax};
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
  // tokens per workgroup: 4, fewer while the launch has less than four
  // workgroups per compute unit; with fewer tokens than that the heads are
  // divided as well (each workgroup then computes the few angles again)
  const int cus = current_cus();
  t.tokens = kMaxTokens;
  while (t.tokens > 1 && (int64_t)args.M < (int64_t)t.tokens * 4 * cus) t.tokens /= 2;
  const int gx = (int)((args.M + t.tokens - 1) / t.tokens);
  const int most = (heads + groups - 1) / groups;  // a head for each lane group at least
  const int gy = std::max(1, std::min(most, (2 * cus) / std::max(1, gx)));
  t.heads_per_wg = (heads + gy - 1) / gy;
  t.heads_magic = (uint32_t)(((1ull << 32) + t.heads_per_wg - 1) / t.heads_per_wg);  // unused for one head
  const dim3 grid(gx, (heads + t.heads_per_wg - 1) / t.heads_per_wg);
  const size_t lds = (size_t)t.tokens * axes.half * sizeof(float2);
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
