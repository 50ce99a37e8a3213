// The 8-bit linear on gfx950: Y = (sum_k q_x q_w) s_x s_w + b with exact int32
// sums, one fp32 scale per token and one per output channel, and an optional
// GELU (tanh form) before the one bf16 rounding.  It serves the projections
// that are kept out of the 4-bit path (mind-verse.de, "Effiziente Optimierung
// von Diffusionsmodellen durch Nunchaku 4-Bit-Quantisierung", section "Nunchaku
// Lite: Nahtlose Integration in Diffusers": precision-sensitive layers).
//
// With no dequantization inside the K loop the kernel is a plain int8 GEMM.  Large
// products are bound by the chip's power: on random codes registers alone feed
// v_mfma_i32_32x32x32_i8 at 3.5 POP/s and v_mfma_i32_16x16x64_i8, which touches its
// accumulators half as often, at 4.05 (both 4.9 on zeros; tests/probes/int8_rate_probe.hip),
// so the second is used, and operands are moved as little as the registers allow.
//  * workgroup tile 32 WI WN weight rows x 32 WJ WM token rows, WN x WM waves of
//    2 WI x 2 WJ tiles of 16 x 16 (256 x 256 on 8 waves: 128 int32 accumulators per
//    lane, two waves per SIMD);
//  * R LDS stages of 128 bytes per row, filled by global_load_lds_dwordx4 with
//    8 whole 128-byte row runs per instruction.  A stage is computed in two
//    halves: while the MFMAs of the first run, the fragments of the second are
//    read; after that the stage's LDS is free, its DMA for stage q + R is
//    issued, and while the second half's MFMAs run the first half of stage
//    q + 1 is read.  One barrier per stage, with R - 1 stages of MFMAs between
//    a DMA and the wait for it;
//  * 16-byte granule g of row R sits at slot 8 R + (g ^ R[3:1]).  A 16-byte LDS
//    read runs in phases of 16 lanes (0-3, 12-15, 20-23, 24-27; 4-11, 16-19, 28-31;
//    the same in the upper half) over 256 bytes of banks: in each phase the even
//    and the odd rows then take 8 different slots, no two lanes one bank;
//  * few tiles: K is split over workgroups, whose int32 partials meet in the
//    caller's workspace (integer sums: the order does not matter).  (The model below does
//    not know of a caller who clears the workspace for each call, as in a captured graph:
//    64 x 12288 -> 3072 12.0 us, captured 13.9);
//  * many tiles: a workgroup stays and takes one after the other; the last R
//    stages of a tile fetch the first of the next, and while its Y leaves they
//    arrive (4608 x 3072 -> 12288 with GELU 165 -> 159 us, 16384 x 4096 -> 4096 221 -> 217).
//    Y with ordinary instead of streaming stores then takes 232 us of the latter,
//    and not waiting for the stores before the next tile's second stage 240: the
//    workgroups of an XCD drift apart and share less of its L2.
//
// The MFMA A operand is the weight tile (rows n), B the token tile (columns m),
// so lane l holds Y[m = l % 16][n = 4 (l / 16) + v] of each 16 x 16 tile; Y leaves
// through LDS in runs of 64 WI bytes per row, 16 rows of a wave at a time (all of a
// wave's rows at once, in the stages' LDS: 1333 x 3072 -> 3072 22.0 us against 19.9).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "row_device.h"
#include "tile_device.h"
#include "w8a8.h"

namespace svdq {
namespace {

struct TileArgs {
  W8a8Args g;
  int splits;    // over K, gridDim.y
  int tiles;     // of the whole launch; without splits a workgroup takes every gridDim.x-th
  u32* count;    // one arrival counter per wave sub-tile (splits > 1)
  int* part;     // int32 partials [sub-tile][splits][WI WJ 16][64]
};

// WN x WM waves of WI x WJ tiles of 32 x 32, R stages in LDS
template <int WI, int WJ, int WN, int WM, int R>
struct Shape {
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int kTN = 32 * WI * WN, kTM = 32 * WJ * WM;
  static constexpr int kLds = R * 128 * (kTN + kTM) + kWaves * 1024 * WI;
  static_assert(kLds <= 160 * 1024, "the stages and the rows of Y on their way fit the LDS");
  static constexpr int kWgs = kLds > 80 * 1024 ? 1 : 2;  // per CU, by LDS
  static constexpr int kSub = WI * WJ * 1024;            // accumulators of a wave
};

// kOne: a tile per workgroup; kSplits: the same over a part of K; kMany: several tiles
// per workgroup, one after the other, all of them whole, K % (128 R) == 0
enum Mode { kOne, kSplits, kMany };

template <int WI, int WJ, int WN, int WM, int R, Mode kMode>
__global__ __launch_bounds__((Shape<WI, WJ, WN, WM, R>::kThreads), 2) void w8a8_tile_kernel(const TileArgs p) {
  using Sh = Shape<WI, WJ, WN, WM, R>;
  static_assert(R >= 2 && R <= 4, "stage buffers");
  constexpr bool kSplit = kMode == kSplits, kWhole = kMode == kMany;
  constexpr int kTN = Sh::kTN, kTM = Sh::kTM, kWaves = Sh::kWaves;
  // one LDS object per operand and stage, so the compiler sees that a DMA
  // into one cannot alias reads of another
  __shared__ __attribute__((aligned(16))) uint8_t w0[kTN * 128], w1[kTN * 128], a0[kTM * 128], a1[kTM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t w2[R > 2 ? kTN * 128 : 16], a2[R > 2 ? kTM * 128 : 16];
  __shared__ __attribute__((aligned(16))) uint8_t w3[R > 3 ? kTN * 128 : 16], a3[R > 3 ? kTM * 128 : 16];
  auto wbuf = [&](int b) -> uint8_t* { return b == 0 ? w0 : b == 1 ? w1 : b == 2 ? w2 : w3; };
  auto abuf = [&](int b) -> uint8_t* { return b == 0 ? a0 : b == 1 ? a1 : b == 2 ? a2 : a3; };

  // the epilogue's own: 16 rows of each wave's sub-tile
  __shared__ __attribute__((aligned(16))) uint8_t rows[kWaves * 1024 * WI];

  const int M = p.g.M, N = p.g.N, K = p.g.K;
  const int tiles_n = (N + kTN - 1) / kTN;
  // stages of 128 k; the last one may be half (K % 128 == 64)
  const int S_all = (K + 127) >> 7;
  const int q_begin = kSplit ? (int)((long)blockIdx.y * S_all / p.splits) : 0;
  const int q_end = kSplit ? (int)((long)(blockIdx.y + 1) * S_all / p.splits) : S_all;
  const bool half_end = q_end == S_all && (K & 64) != 0;
  const int S = q_end - q_begin - (half_end ? 1 : 0);  // whole stages

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / WM;
  const int wm = wave % WM;
  const int l16 = lane & 15;
  const int lq = lane >> 4;

  // DMA role: instruction k of a wave fills rows 8 (waves k + wave) + lane / 8, slot
  // lane % 8 of each row, with granule (lane % 8) ^ row[3:1].  Rows past the
  // end repeat the last row (never stored).  In a half stage the granules of
  // the missing half repeat those of the first.
  const u32 gran = 16u * (u32)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
  const u32 back = !kWhole && (K & 64) != 0 && gran >= 64 ? 64u : 0u;
  constexpr int kWd = kTN / (8 * kWaves), kAd = kTM / (8 * kWaves);  // DMAs per stage and wave
  static_assert(kWaves % 2 == 0 && kWd * 8 * kWaves == kTN && kAd * 8 * kWaves == kTM, "whole row runs per wave");
  const u32 wlane = (u32)(lane >> 3) * (u32)K + gran;
  const uint8_t *wbase, *abase;
  u32 woff[kWd], aoff[kAd];
  // the tile that the DMAs fill (one or more stages ahead of the products)
  int n0, m0;
  auto dma_tile = [&](int t) {
    int tm, tn;
    tile_of(t, (M + kTM - 1) / kTM, tiles_n, tm, tn);
    n0 = tn * kTN, m0 = tm * kTM;
    wbase = reinterpret_cast<const uint8_t*>(p.g.w) + (size_t)n0 * (size_t)K;
    abase = reinterpret_cast<const uint8_t*>(p.g.act) + (size_t)m0 * (size_t)K;
    // (N % 64 == 0: the 8 weight rows of an instruction are all inside or all
    // past the end, so their offset is uniform)
#pragma unroll
    for (int k = 0; k < kWd; ++k) {
      const int row = 8 * (kWaves * k + wave);
      woff[k] = (u32)(kWhole ? row : __builtin_amdgcn_readfirstlane(min(n0 + row, N - 8) - n0)) * (u32)K;
    }
#pragma unroll
    for (int k = 0; k < kAd; ++k) {
      const int row = 8 * (kWaves * k + wave);
      if constexpr (kWhole) aoff[k] = (u32)row * (u32)K;
      else aoff[k] = (u32)(min(m0 + row + (lane >> 3), M - 1) - m0) * (u32)K + gran;
    }
  };
  // column of stage q (counted from q_begin; past the end the last stage again), and
  // how far back the lane's granule lies in it
  auto stage_col = [&](int q) {
    const int s = min(q_begin + q, q_end - 1);
    return u32x2{128u * (u32)s, s == S_all - 1 ? back : 0u};
  };
  constexpr int kDmas = kWd + kAd;
  auto dma_one = [&](int k, u32x2 col, u32 wlane, auto bc) {
    constexpr int b = decltype(bc)::value;
    const int ka = k - kWd;
    if (k < kWd) dma16(wbase + (woff[k] + col.x) + (wlane - col.y), wbuf(b) + 1024 * (kWaves * k + wave));
    else if constexpr (kWhole) dma16(abase + (aoff[ka] + col.x) + wlane, abuf(b) + 1024 * (kWaves * ka + wave));
    else dma16(abase + col.x + (aoff[ka] - col.y), abuf(b) + 1024 * (kWaves * ka + wave));
  };
  auto dma_stage = [&](int q, auto bc) {
    const u32x2 col = stage_col(q);
#pragma unroll
    for (int k = 0; k < kDmas; ++k) dma_one(k, col, wlane, bc);
  };

  // Fragment reads: lane (l16, lq) takes granule 4 hh + lq of rows 16 i + l16 for
  // half hh, a k step of 64.
  constexpr int kI = 2 * WI, kJ = 2 * WJ;  // 16 x 16 tiles of a wave
  const int fo = 128 * l16 + 16 * (lq ^ (l16 >> 1));
  const int wrow = wn * 32 * WI * 128, arow = wm * 32 * WJ * 128;
  struct Frags {
    v4i w[kI], a[kJ];
  };
  auto read_half = [&](Frags& f, auto bc, auto hc) {
    constexpr int b = decltype(bc)::value, hh = decltype(hc)::value;
    const uint8_t* wt = wbuf(b) + wrow;
    const uint8_t* at = abuf(b) + arow;
    int at0 = fo;
    __asm__ volatile("" : "+v"(at0));  // no register per buffer and half
    at0 ^= 64 * hh;
#pragma unroll
    for (int i = 0; i < kI; ++i) f.w[i] = *reinterpret_cast<const v4i*>(wt + at0 + 2048 * i);
#pragma unroll
    for (int j = 0; j < kJ; ++j) f.a[j] = *reinterpret_cast<const v4i*>(at + at0 + 2048 * j);
  };

  v4i acc[kI][kJ];
  auto mfma_half = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[i], f.a[j], acc[i][j], 0, 0, 0);
  };
  // One LDS read (two where there are more of them than MFMAs) after each of
  // the first MFMAs of a half; in the second half the DMAs are spread over the
  // MFMAs, so that the waves do not queue for the address unit while the matrix
  // core idles.
  auto interleave = [&](auto with_dma) {
    constexpr int kReads = kI + kJ, kMfmas = kI * kJ;
    constexpr int kRead = (kReads + kMfmas - 1) / kMfmas;
    constexpr int kEvery = kMfmas / kDmas > 0 ? kMfmas / kDmas : 1, kDma = (kDmas * kEvery + kMfmas - 1) / kMfmas;
#pragma unroll
    for (int k = 0; k < kMfmas; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (k * kRead < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kRead, 0);
      if constexpr (decltype(with_dma)::value)
        if (k % kEvery == kEvery - 1) __builtin_amdgcn_sched_group_barrier(0x020, kDma, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  using B0 = std::integral_constant<int, 0>;
  using B1 = std::integral_constant<int, 1>;
  using B2 = std::integral_constant<int, 2>;
  using B3 = std::integral_constant<int, 3>;
  Frags f0, f1;
  int shift = 0;  // stages by which the DMAs run ahead into the next tile
  auto iteration = [&](int q, auto bc) {
    constexpr int b = decltype(bc)::value;
    using BC = std::integral_constant<int, b>;
    using BN = std::integral_constant<int, (b + 1) % R>;
    __builtin_amdgcn_sched_barrier(0);
    read_half(f1, BC{}, B1{});
    mfma_half(f0);
    interleave(B0{});
    const u32x2 col = stage_col(q + R + shift);
    // this wave's reads of the stage, and its DMAs of the next one; those of
    // the R - 2 stages after it may still be in flight
    wait_vm_lds<(R - 2) * kDmas>();
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_half(f0, BN{}, B0{});
    u32 wl = wlane;
    if constexpr (kWhole) __asm__ volatile("" : "+v"(wl));  // a 32-bit offset to a uniform address
#pragma unroll
    for (int k = 0; k < kDmas; ++k) dma_one(k, col, wl, bc);
    mfma_half(f1);
    interleave(B1{});
  };
  int tile = blockIdx.x;
  dma_tile(tile);
  dma_stage(0, B0{});
  dma_stage(1, B1{});
  if constexpr (R > 2) dma_stage(2, B2{});
  if constexpr (R > 3) dma_stage(3, B3{});
  wait_vm_lds<(R - 1) * kDmas>();
  barrier();
  for (;;) {
    read_half(f0, B0{}, B0{});
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    const int tn0 = n0, tm0 = m0;  // of the products
    const int next = tile + (int)gridDim.x;
    const bool more = kWhole && next < p.tiles;
    shift = 0;
    int q = 0;
    for (; q + R <= S; q += R) {
      // the last R stages fetch the first of the next tile
      if (more && q + R == S) {
        dma_tile(next);
        shift = -S;
      }
      iteration(q, B0{});
      iteration(q + 1, B1{});
      if constexpr (R > 2) iteration(q + 2, B2{});
      if constexpr (R > 3) iteration(q + 3, B3{});
    }
    if constexpr (!kWhole) {
      if (q < S) iteration(q, B0{});
      if constexpr (R > 2)
        if (q + 1 < S) iteration(q + 1, B1{});
      if constexpr (R > 3)
        if (q + 2 < S) iteration(q + 2, B2{});
      if (half_end) mfma_half(f0);
    }

    if constexpr (kSplit) {
      // Each wave stores its int32 sub-tile with agent-coherent stores, waits
      // for them and bumps the sub-tile's counter (which wraps to zero); the
      // last to arrive adds the others' and runs the epilogue.
      constexpr int kSub = Sh::kSub;
      const size_t sub = (size_t)tile * kWaves + wave;
      int* mine = p.part + (sub * p.splits + blockIdx.y) * kSub + lane;
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            __hip_atomic_store(mine + (((i * kJ + j) * 4 + e) << 6), acc[i][j][e], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
      __asm__ volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): the partial is visible to the agent
      __asm__ volatile("" ::: "memory");
      u32 old = 0;
      if (lane == 0) old = atomicInc(p.count + sub, (u32)(p.splits - 1));
      old = __shfl(old, 0);
      if (old != (u32)(p.splits - 1)) break;
      __asm__ volatile("" ::: "memory");
      for (int s = 0; s < p.splits; ++s) {
        if (s == (int)blockIdx.y) continue;
        const int* src = p.part + (sub * p.splits + s) * kSub + lane;
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          v4i t[kJ];
#pragma unroll
          for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              t[j][e] = __hip_atomic_load(src + (((i * kJ + j) * 4 + e) << 6), __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
          for (int j = 0; j < kJ; ++j) acc[i][j] += t[j];
        }
      }
    }

    // y = bf16(epi(acc fl32(s_x s_w) + b)) in fp32 (int32 -> fp32 rounds to 24
    // bits, far below the bf16 rounding).  The wave turns its sub-tile 16 token rows
    // at a time through LDS of its own, so that Y leaves in row runs of 64 WI bytes.
    constexpr int kChunks = 4 * WI;                    // 16-byte chunks of a sub-tile row
    constexpr int kMask = kChunks % 8 == 0 ? 7 : 3;    // chunk c of row m sits at c ^ (m & kMask)
    // (the lane number anew: what the epilogue derives from it is not worth
    // registers during the products)
    int el = lane;
    __asm__ volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(el));
    const int e16 = el & 15, eq = el >> 4;
    uint8_t* turn = rows + wave * 1024 * WI;
    const int nw = tn0 + wn * 32 * WI, mw = tm0 + wm * 32 * WJ;  // the wave's first column and row
    float sx[kJ];
    float4 sw[kI];
    uint2 b2[kI];
#pragma unroll
    for (int j = 0; j < kJ; ++j) sx[j] = p.g.act_scales[kWhole ? mw + 16 * j + e16 : min(mw + 16 * j + e16, M - 1)];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int nc = kWhole ? nw + 16 * i + 4 * eq : min(nw + 16 * i + 4 * eq, N - 4);
      sw[i] = *reinterpret_cast<const float4*>(p.g.w_scales + nc);
      b2[i] = p.g.bias != nullptr ? *reinterpret_cast<const uint2*>(p.g.bias + nc) : uint2{0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        float o[4];
        o[0] = __builtin_fmaf((float)acc[i][j][0], sx[j] * sw[i].x, bf16_lo(b2[i].x));
        o[1] = __builtin_fmaf((float)acc[i][j][1], sx[j] * sw[i].y, bf16_hi(b2[i].x));
        o[2] = __builtin_fmaf((float)acc[i][j][2], sx[j] * sw[i].z, bf16_lo(b2[i].y));
        o[3] = __builtin_fmaf((float)acc[i][j][3], sx[j] * sw[i].w, bf16_hi(b2[i].y));
        if (p.g.epilogue == kEpilogueGelu) {
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = gelu_exp2(o[v]);
        }
        const int nl = 16 * i + 4 * eq;  // within the wave's columns
        uint8_t* dst = turn + e16 * (16 * kChunks) + (((nl >> 3) ^ (e16 & kMask)) << 4) + 8 * (eq & 1);
        *reinterpret_cast<uint2*>(dst) = uint2{pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3])};
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes are done
      __asm__ volatile("" ::: "memory");
      // chunk by chunk in row order: an instruction stores 64 chunks, whole rows of
      // 64 WI bytes where they divide 64
#pragma unroll
      for (int t = 0; t < WI; ++t) {
        const int at = 64 * t + el;
        const int ml = at / kChunks, c = at - ml * kChunks;
        const int m = mw + 16 * j + ml, n = nw + 8 * c;
        const uint4 v = *reinterpret_cast<const uint4*>(turn + ml * (16 * kChunks) + ((c ^ (ml & kMask)) << 4));
        // streaming (non-temporal) stores: Y is not read again by this launch;
        // N % 64 == 0, so n < N covers n + 7
        if (kWhole || (m < M && n < N))
          __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p.g.y + (size_t)m * N + n));
      }
      __asm__ volatile("" ::: "memory");  // (a wave's LDS operations run in order)
    }
    if (!more) break;
    tile = next;
  }
  wait_vm_lds<0>();  // no DMA may land after the workgroup's end
}

struct Plan {
  int shape;    // index into kShapes
  int tiles;
  int splits;
  double cost;  // us, by the model below
};

// Workgroup tiles, the test hook's name of each (channels / 64, tokens / 64, LDS
// stages) and what a launch of it takes: with n workgroups on the busiest
// compute unit, base + n (fill + S step) us for S stages of 128 k; where two
// workgroups share a compute unit, base + (n / 2) (fill2 + S step2), an odd one
// at fill and step.  Fitted to 80 shapes (65 to 4608 tokens, K 512 to 12288, N 256
// to 12288) on MI355X, every tile and split timed: the plan's pick is within 0.3 %
// (geometric mean) of the best measured one, 6 % at most.
#define SVDQ_SHAPES(X)                                   \
  X(442, 4, 2, 2, 4, 2, -3.29, 11.18, 1.109, 0.0, 0.0)   \
  X(342, 3, 2, 2, 4, 2, -2.66, 9.36, 0.937, 0.0, 0.0)    \
  X(432, 2, 3, 4, 2, 2, -1.86, 8.15, 0.941, 0.0, 0.0)    \
  X(323, 3, 2, 2, 2, 3, 0.14, 6.64, 0.507, 0.0, 0.0)     \
  X(224, 2, 2, 2, 2, 4, 1.06, 4.89, 0.372, 0.0, 0.0)     \
  X(222, 2, 2, 2, 2, 2, 0.66, 3.67, 0.619, 5.38, 0.788)  \
  X(124, 1, 2, 2, 2, 4, 2.08, 2.83, 0.260, 0.0, 0.0)     \
  X(114, 1, 1, 2, 2, 4, 3.00, 1.45, 0.175, 2.07, 0.365)
struct ShapeInfo {
  int code, tn, tm, waves, wgs, sub;
  double base, fill, step, fill2, step2;
};
template <int WI, int WJ, int WN, int WM, int R>
constexpr ShapeInfo info(int code, double base, double fill, double step, double fill2, double step2) {
  using S = Shape<WI, WJ, WN, WM, R>;
  return ShapeInfo{code, S::kTN, S::kTM, S::kWaves, S::kWgs, S::kSub, base, fill, step, fill2, step2};
}
#define SVDQ_INFO(code, wi, wj, wn, wm, r, base, fill, step, fill2, step2) \
  info<wi, wj, wn, wm, r>(code, base, fill, step, fill2, step2),
constexpr ShapeInfo kShapes[] = {SVDQ_SHAPES(SVDQ_INFO)};
#undef SVDQ_INFO
constexpr int kMaxSplits = 16;

std::atomic<int> g_tile{0}, g_splits{0};  // test hook

// the cheapest tile and K-split
Plan plan_of(int64_t M, int64_t N, int64_t K) {
  const int cus = current_cus();
  const int stages = (int)((K + 127) / 128);
  const int forced_tile = g_tile.load(std::memory_order_relaxed), forced = g_splits.load(std::memory_order_relaxed);
  Plan best{-1, 0, 1, 0.0};
  for (int i = 0; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i) {
    const ShapeInfo& s = kShapes[i];
    if (forced_tile > 1 && forced_tile != s.code) continue;
    const int64_t tiles = ((N + s.tn - 1) / s.tn) * ((M + s.tm - 1) / s.tm);
    if (tiles > (1 << 30)) continue;
    for (int splits = 1; splits <= std::min(kMaxSplits, stages); splits *= 2) {
      const int64_t wgs = tiles * splits;
      if (splits > 1 && tiles * s.waves > (int64_t)kWsMaxCounters) break;
      if (forced > 0 ? splits > forced : splits > 1 && wgs > 2 * cus) break;
      const double n = (double)((wgs + cus - 1) / cus), S = (double)((stages + splits - 1) / splits);
      double cost = s.base;
      if (s.wgs == 2) {
        const double pairs = std::floor(n / 2);
        cost += pairs * (s.fill2 + S * s.step2) + (n - 2 * pairs) * (s.fill + S * s.step);
      } else {
        cost += n * (s.fill + S * s.step);
      }
      if (splits > 1) cost += 2.54 + 0.52 * splits + 0.57 * (s.tn / 64) * (s.tm / 64);  // the partials' round trips
      if (best.shape < 0 || cost < best.cost || (forced > 0 && best.shape == i)) best = Plan{i, (int)tiles, splits, cost};
    }
  }
  return best;
}

// The launches of a product: the tokens [0, m1) in whole rounds of one of the
// largest tiles, and the rest on the tile that suits it (m1 = M: one launch).  The
// last round of a large tile otherwise leaves most compute units idle (4608 tokens,
// 3072 -> 12288: 864 tiles of 256 x 256 are 3.4 rounds, 156 us; 768 and then 256 of 192 x 128
// are 4 full ones, the last of them a short one, 150 us).
// kSecondLaunch: what a second launch takes beyond the model's sum, in us (of 15
// shapes where the two come close, 3 then run longer than the other choice, by 5 % at most).
constexpr double kSecondLaunch = 6.5;
struct Launches {
  int64_t m1;
  Plan first, rest;
};
Launches launches_of(int64_t M, int64_t N, int64_t K) {
  Launches best{M, plan_of(M, N, K), Plan{}};
  if (g_tile.load(std::memory_order_relaxed) > 1 || g_splits.load(std::memory_order_relaxed) > 0) return best;
  const int cus = current_cus();
  const double S = (double)((K + 127) / 128);
  double best_cost = best.first.cost;
  for (int i = 0; i < 3; ++i) {
    const ShapeInfo& s = kShapes[i];
    const int64_t nt = (N + s.tn - 1) / s.tn, mt = (M + s.tm - 1) / s.tm;
    const int64_t rounds = nt * mt / cus, mt1 = rounds * cus / nt;
    if (nt * mt > (1 << 30) || mt1 <= 0 || mt1 * s.tm >= M) continue;
    Launches l{mt1 * s.tm, Plan{i, (int)(mt1 * nt), 1, 0.0}, plan_of(M - mt1 * s.tm, N, K)};
    l.first.cost = kSecondLaunch + s.base + (double)((mt1 * nt + cus - 1) / cus) * (s.fill + S * s.step);
    if (l.first.cost + l.rest.cost < best_cost) {
      best = l;
      best_cost = l.first.cost + l.rest.cost;
    }
  }
  return best;
}

template <int WI, int WJ, int WN, int WM, int R>
void tile_go(const TileArgs& t, int tiles, hipStream_t stream) {
  using Sh = Shape<WI, WJ, WN, WM, R>;
  const dim3 block(Sh::kThreads);
  // whole tiles, more than the chip holds at once: one workgroup per compute unit
  // (of the large tiles, which the plan takes for such products)
  if constexpr (Sh::kWaves == 8) {
    const int cus = current_cus();
    if (t.splits == 1 && tiles > cus && t.g.M % Sh::kTM == 0 && t.g.N % Sh::kTN == 0 && t.g.K % (128 * R) == 0) {
      hipLaunchKernelGGL((w8a8_tile_kernel<WI, WJ, WN, WM, R, kMany>), dim3(cus), block, 0, stream, t);
      return;
    }
  }
  if (t.splits > 1)
    hipLaunchKernelGGL((w8a8_tile_kernel<WI, WJ, WN, WM, R, kSplits>), dim3(tiles, t.splits), block, 0, stream, t);
  else
    hipLaunchKernelGGL((w8a8_tile_kernel<WI, WJ, WN, WM, R, kOne>), dim3(tiles), block, 0, stream, t);
}

}  // namespace

bool w8a8_tile_known(int tile) {
  if (tile == 0 || tile == 1) return true;
  for (const ShapeInfo& s : kShapes)
    if (s.code == tile) return true;
  return false;
}

void set_w8a8_plan_override(int tile, int splits) {
  g_tile.store(tile, std::memory_order_relaxed);
  g_splits.store(splits, std::memory_order_relaxed);
}

// The weight-streaming kernel for up to 4 tokens, and up to 16 where its workgroups
// (one per 16 channels) are fewer than two per compute unit.  Measured, it against the
// best tile, in a graph, the weights from HBM: 1 token 3072 -> 3072 4.9 / 7.9 us, 3072 -> 12288
// 9.3 / 10.7, 12288 -> 3072 11.0 / 13.0; 4 tokens 5.1 / 8.0, 10.1 / 10.8, 11.6 / 13.1; 16 tokens
// 6.3 / 8.1, 13.8 / 11.0, 16.8 / 13.3 (the rule does not look at K: with a long one the
// tiles are the quicker from 9 tokens or so, where they need no cleared workspace).
static bool few_tokens(int64_t M, int64_t N) {
  const int t = g_tile.load(std::memory_order_relaxed);
  return t == 1 ? M <= 16 : t == 0 && (M <= 4 || (M <= 16 && N / 16 < 2 * current_cus()));
}

static size_t plan_bytes(const Plan& p) {
  if (p.splits <= 1) return 0;
  const ShapeInfo& s = kShapes[p.shape];
  return ws_bytes((size_t)p.tiles * s.waves, (size_t)p.tiles * s.waves * p.splits * s.sub * sizeof(int));
}

size_t w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (few_tokens(M, N)) return 0;
  const Launches l = launches_of(M, N, K);
  return std::max(plan_bytes(l.first), l.m1 < M ? plan_bytes(l.rest) : 0);
}

static hipError_t launch_plan(const W8a8Args& a, const Plan& p, const Workspace& ws, hipStream_t stream) {
  if (plan_bytes(p) > ws.bytes) return hipErrorInvalidValue;
  TileArgs t{a, p.splits, p.tiles, nullptr, nullptr};
  if (p.splits > 1) {
    t.count = ws_counters(ws);
    t.part = static_cast<int*>(ws_scratch(ws));
  }
  switch (kShapes[p.shape].code) {
#define SVDQ_GO(code, wi, wj, wn, wm, r, base, fill, step, fill2, step2) \
  case code: tile_go<wi, wj, wn, wm, r>(t, p.tiles, stream); break;
    SVDQ_SHAPES(SVDQ_GO)
#undef SVDQ_GO
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_w8a8_gemm(const W8a8Args& a, Workspace ws, hipStream_t stream) {
  if (few_tokens(a.M, a.N)) return launch_w8a8_skinny(a, stream);
  const Launches l = launches_of(a.M, a.N, a.K);
  W8a8Args part = a;
  part.M = (int)l.m1;
  const hipError_t e = launch_plan(part, l.first, ws, stream);
  if (e != hipSuccess || l.m1 == a.M) return e;
  part.M = (int)(a.M - l.m1);
  part.act += (size_t)l.m1 * (size_t)a.K;
  part.act_scales += l.m1;
  part.y += (size_t)l.m1 * (size_t)a.N;
  return launch_plan(part, l.rest, ws, stream);
}

}  // namespace svdq
