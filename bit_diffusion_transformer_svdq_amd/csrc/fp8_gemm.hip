// The 8-bit floating-point linear on gfx950:
//   Y[m,n] = epi( sum_b s_x[b,m] s_w[n/128,b] (sum_{k in b} q_x[m,k] q_w[n,k]) + bias[n] )
// over blocks b of 128 channels, e4m3 codes, and its gated form, two such products of
// the same tokens, H = act(G) U, as bf16 or as the next linear's codes.
//
// A block is exactly the K of one v_mfma_f32_16x16x128_f8f6f4 (32 cycles, 2048 operations
// a cycle and SIMD): every MFMA starts from zero and its four results per lane join the
// fp32 sums by one fma each with the block's scale.  (From registers, two waves per SIMD, on
// zero codes, an MFMA with its 4 fmas takes 1.11 times as long as one alone, 35.4 cycles
// (profiles/rates_fp8_operators.txt): the vector unit works beside the matrix core, with
// little to spare for anything but the fmas.)  With the weights as the A
// operand a lane's results belong to one token, so the scale s_x s_w is one product per
// token tile and block, not one per result.
//
// The matrix core adds e4m3 products eight neighbours along K at a time, each cut off (towards
// zero) below 2^-13 of 2^r, r the largest sum of two codes' exponents among the eight; it
// adds the groups' sums in fp32 (tests/probes/e4m3_sum_probe.hip).  Every MFMA that takes e4m3
// does so.  A product of two codes has 8 significant bits, so only those smaller than 2^-7 of the
// group's largest lose any: before the bf16 rounding of Y (1.7e-3 on average) it does not
// show, but 0.35 % of the codes of an H are the neighbours of those that exact sums give (a whole
// feed-forward block is 2.1e-3 to 2.6e-3 from the exact result, 1.7e-3 with fp32 products:
// profiles/fp8_h_codes.txt).
//  * workgroup tile of WN x WM waves, each 32 H weight rows x 16 J token rows (256 x 256 on
//    8 waves, H = J = 4: 128 fp32 sums per lane, two waves per SIMD); weight rows come in
//    two halves, in the gated form G's and U's of the same features, so that H is
//    formed in registers;
//  * R LDS stages of 128 bytes per row, filled by global_load_lds_dwordx4; a row's
//    granule g of 16 bytes sits at slot g ^ row[3:1] (bank conflicts: see
//    w8a8_gemm.hip), token scales beside them.  A lane takes granules lq and lq + 4 of its
//    rows: the order within a block does not matter as long as both operands have it;
//  * a stage is computed in phases of 2 x J tiles.  While a phase's MFMAs run, the weight
//    fragments of the next are read; in the last one, behind a barrier, the next stage's
//    tokens take the places of this one's as they are used up, and the stage's LDS, read
//    by all, is filled for stage q + R;
//  * results join kLag slots after their MFMA and MFMAs come ahead of their slot's fmas
//    (2 slots, in any order: 4096 x 8192 -> 4096 123 us against 112);
//  * few tiles: K is split over workgroups, whose fp32 partials meet in the caller's
//    workspace; the last to arrive adds them in the order of K, so that results do
//    not depend on timing;
//  * many tiles: a workgroup stays and takes one after the other, as in w8a8_gemm.hip.
//
// 8192^3 takes 2.5 PFLOP/s and 4096 x 8192 -> 4096 108-113 us, 2.4-2.5; with all codes zero 80 us:
// on random codes large products are bound by the chip's power (the clock falls from 2.3
// to 2.0 GHz), otherwise by the MFMAs and fmas.  The second one without the stages' loads 94 us
// (zero codes 74), without the LDS reads 101 (78), without both 88 (71): what is left are the MFMAs,
// fmas, barriers and Y.  A round of 256 x 256 tiles on all compute units takes 1.65 us per stage
// and 6 to 7 us for its Y, which all of them write at once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "fp8.h"
#include "tile_device.h"

namespace svdq {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void dma4(const void* gptr, uint8_t* lds_wave_base) {
  __builtin_amdgcn_global_load_lds((glb_void*)gptr, (lds_void*)lds_wave_base, 4, 0, 0);
}

struct TileArgs {
  Fp8Args g;
  int splits;   // over K, gridDim.y
  int tiles;    // of the whole launch
  u32* count;   // one arrival counter per tile (splits > 1)
  float* part;  // fp32 partials [tile][splits][waves][2 H J][64][4]
};

// WN x WM waves of 2 H x J tiles of 16 x 16, R stages in LDS
template <int H, int J, int WN, int WM, int R>
struct Shape {
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int kTN = 32 * H * WN, kTM = 16 * J * WM;
  static constexpr int kTurn = 512 * H;  // bytes of 16 rows of a wave's columns on their way out
  static constexpr int kLds = R * (128 * (kTN + kTM) + 4 * kTM) + kWaves * kTurn;
  static_assert(kLds <= 160 * 1024 - 1024, "the stages and the rows of Y on their way fit the LDS");
  static constexpr int kWgs = kLds > 79 * 1024 ? 1 : 2;  // per CU, by LDS
};

enum Form { kPlain, kGated, kGatedCodes };
// kOne: a tile per workgroup; kSplits: the same over a part of K; kMany: several tiles
// per workgroup, one after the other, all of them whole, ceil(K / 128) % R == 0
enum Mode { kOne, kSplits, kMany };

template <int H, int J, int WN, int WM, int R, Form kForm, Mode kMode>
__global__ __launch_bounds__((Shape<H, J, WN, WM, R>::kThreads), 2) void fp8_tile_kernel(const TileArgs p) {
  using Sh = Shape<H, J, WN, WM, R>;
  static_assert(R >= 2 && R <= 4, "stage buffers");
  constexpr bool kSplit = kMode == kSplits, kWhole = kMode == kMany;
  constexpr bool kGate = kForm != kPlain;
  constexpr int kTN = Sh::kTN, kTM = Sh::kTM, kWaves = Sh::kWaves;
  constexpr int kCols = kGate ? kTN / 2 : kTN;        // output columns of a tile
  constexpr int kWaveCols = kGate ? 16 * H : 32 * H;  // and of a wave
  // one LDS object per operand (per half of the weight rows) and stage, so the compiler
  // sees that a DMA into one cannot alias reads of another
#define SVDQ_STAGE(b)                                                                                            \
  __shared__ __attribute__((aligned(16))) uint8_t g##b[R > b ? kTN * 64 : 16], u##b[R > b ? kTN * 64 : 16],      \
      a##b[R > b ? kTM * 128 : 16], s##b[R > b ? kTM * 4 : 16];
  SVDQ_STAGE(0) SVDQ_STAGE(1) SVDQ_STAGE(2) SVDQ_STAGE(3)
#undef SVDQ_STAGE
#define SVDQ_PICK(x) b == 0 ? x##0 : b == 1 ? x##1 : b == 2 ? x##2 : x##3
  // the first half of the waves' weight rows, 16 H of each wave (gated: G's), and the second
  auto wbuf = [&](int b, int half) -> uint8_t* { return half == 0 ? (SVDQ_PICK(g)) : (SVDQ_PICK(u)); };
  auto abuf = [&](int b) -> uint8_t* { return SVDQ_PICK(a); };
  auto sbuf = [&](int b) -> uint8_t* { return SVDQ_PICK(s); };
#undef SVDQ_PICK
  __shared__ __attribute__((aligned(16))) uint8_t rows[kWaves * Sh::kTurn];  // the epilogue's own
  __shared__ float red[kForm == kGatedCodes ? kWaves * 16 * J : 1];
  __shared__ u32 arrived;

  const int M = p.g.M, N = p.g.N, K = p.g.K;
  const int tiles_n = (N + kCols - 1) / kCols;
  const int S_all = (K + 127) >> 7;  // stages; the last one may be half (K % 128 == 64)
  const int q_begin = kSplit ? (int)((long)blockIdx.y * S_all / p.splits) : 0;
  const int q_end = kSplit ? (int)((long)(blockIdx.y + 1) * S_all / p.splits) : S_all;
  const int S = q_end - q_begin;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / WM;
  const int wm = wave % WM;
  const int l16 = lane & 15;
  const int lq = lane >> 4;
  // Weight scales of the wave's two halves, one of each a stage, by scalar loads (as
  // constant memory: nothing writes them during the launch) a stage ahead
  typedef const float __attribute__((address_space(4))) cfloat;
  cfloat *ws0, *ws1;
  float sw0, sw1;
  // the half stage sums its 64 products twice (below) and halves the weights' scale, which
  // is exact but for odd multiples of 2^-149 below 2^-125.  (Halving s_x s_w is always exact
  // and took 1 % of the large products, zeros in the tokens' registers made the largest tile spill.)
  const int half_at = q_end == S_all && (K & 64) != 0 ? S - 1 : S;
  auto load_ws = [&](int q) {
    const int at = min(q, S - 1);
    sw0 = ws0[at];
    if constexpr (kGate) sw1 = ws1[at];
  };

  // DMA role: instruction k of a wave fills rows 8 (waves k + wave) + lane / 8, slot
  // lane % 8 of each row, with granule (lane % 8) ^ row[3:1].  Rows past the
  // end repeat the last row (never stored).  In a half stage the granules of
  // the missing half repeat those of the first, in both operands: the sum is twice that of
  // the 64 products, its scale is halved.
  const u32 gran = 16u * (u32)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
  const u32 back = (K & 64) != 0 && gran >= 64 ? 64u : 0u;
  constexpr int kWd = kTN / (8 * kWaves), kAd = kTM / (8 * kWaves);  // DMAs per stage and wave
  constexpr int kDmas = kWd + kAd + 1;                               // and one of the token scales
  static_assert(kWaves % 2 == 0 && kWd % 2 == 0 && kWd * 8 * kWaves == kTN && kAd * 8 * kWaves == kTM, "whole row runs per wave");
  static_assert(kTM % 64 == 0 && kTM <= 64 * kWaves, "the waves cover the token scales");
  const u32 wlane = (u32)(lane >> 3) * (u32)K + gran;
  const uint8_t *abase, *sbase;
  const uint8_t* wbase[2];  // of each half
  u32 woff[kWd], aoff[kAd], soff;
  const int srow = 64 * (wave % (kTM / 64));  // the wave's run of token scales
  // the tile that the DMAs fill (one or more stages ahead of the products)
  int tn, n0, m0;
  auto dma_tile = [&](int t) {
    int tm;
    tile_of(t, (M + kTM - 1) / kTM, (N + kCols - 1) / kCols, tm, tn);
    n0 = tn * kCols, m0 = tm * kTM;
    abase = p.g.act + (size_t)m0 * (size_t)K;
    sbase = reinterpret_cast<const uint8_t*>(p.g.act_scales + m0);
    // (N % 64 == 0: the 8 weight rows of an instruction are all inside or all
    // past the end, so their address is uniform)
    wbase[0] = p.g.w + (size_t)n0 * (size_t)K;
    wbase[1] = kGate ? p.g.up + (size_t)n0 * (size_t)K : wbase[0];
#pragma unroll
    for (int k = 0; k < kWd; ++k) {
      const bool second = k >= kWd / 2;
      const int row = 8 * (kWaves * (second ? k - kWd / 2 : k) + wave);  // of the half
      const int n = kGate ? row : row / (16 * H) * (32 * H) + row % (16 * H) + (second ? 16 * H : 0);
      woff[k] = (u32)(kWhole ? n : min(n0 + n, N - 8) - n0) * (u32)K;
    }
  };
  auto lane_offsets = [&] {
#pragma unroll
    for (int k = 0; k < kAd; ++k) {
      const int row = 8 * (kWaves * k + wave) + (lane >> 3);
      aoff[k] = (u32)(kWhole ? row : min(m0 + row, M - 1) - m0) * (u32)K + gran;
    }
    soff = 4u * (u32)(kWhole ? srow + lane : min(m0 + srow + lane, M - 1) - m0);
  };
  struct Col {
    u32 x, back;
    const uint8_t* s;
  };
  // column of stage q (counted from q_begin; past the end the last stage again)
  auto stage_col = [&](int q) {
    const int s = min(q_begin + q, q_end - 1);
    return Col{128u * (u32)s, s == S_all - 1 ? back : 0u, sbase + 4 * (size_t)s * (size_t)p.g.act_stride};
  };
  // DMA k of a stage: the first half of the weights, tokens, token scales, the second half
  auto dma_one = [&](int k, const Col& col, auto bc) {
    constexpr int b = decltype(bc)::value, h = kWd / 2;
    if (k < h) dma16(wbase[0] + (woff[k] + col.x) + (wlane - col.back), wbuf(b, 0) + 1024 * (kWaves * k + wave));
    else if (k < h + kAd)
      dma16(abase + col.x + (aoff[k - h] - col.back), abuf(b) + 1024 * (kWaves * (k - h) + wave));
    else if (k == h + kAd) dma4(col.s + soff, sbuf(b) + 4 * srow);
    else
      dma16(wbase[1] + (woff[k - kAd - 1] + col.x) + (wlane - col.back), wbuf(b, 1) + 1024 * (kWaves * (k - h - kAd - 1) + wave));
  };
  // With two stages of four phases (kTwice) a stage's LDS is given back in two parts: its
  // tokens and the first half of its weights have been read when its second phase begins,
  // the rest when the last one does.  So every DMA has a stage and a half to arrive (in one
  // part, a stage: 4096 x 8192 -> 4096 116 us against 114.)
  constexpr bool kTwice = H == 4 && R == 2;
  constexpr int kLate = kTwice ? kWd / 2 : 0, kEarly = kDmas - kLate;
  auto dma_stage = [&](int q, auto bc) {
    const Col col = stage_col(q);
#pragma unroll
    for (int k = 0; k < kDmas; ++k) dma_one(k, col, bc);
  };

  // Fragments: lane (l16, lq) takes granules lq and lq + 4 of row 16 i + l16.
  // The smaller tiles of an even number of stages take a whole stage's fragments a stage
  // ahead of its MFMAs (kAhead), so that one phase and one trip to LDS remain per stage.
  constexpr bool kAhead = H <= 2 && R % 2 == 0;
  constexpr int kG = kAhead ? 2 * H : H > 1 ? 2 : 1;  // weight tiles of a phase
  constexpr int kP = 2 * H / kG;          // phases of a stage; the first half of them is the first half of the rows
  constexpr int kSlots = kG * J;          // MFMAs of a phase
  const int fo = 128 * l16 + 16 * (lq ^ (l16 >> 1));
  const int wrow = wn * 16 * H * 128, arow = wm * 16 * J * 128;
  v8i fw[2][kG], fa[kAhead ? 2 : 1][J];
  float st[J];
  // (the address anew for each phase: registers for every buffer's are worth more)
  auto at_row = [&] {
    int at = fo;
    __asm__ volatile("" : "+v"(at));
    return at;
  };
  auto read_tile = [&](const uint8_t* t, int at) {
    const v4i lo = *reinterpret_cast<const v4i*>(t + at), hi = *reinterpret_cast<const v4i*>(t + (at ^ 64));
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto read_w = [&](auto bc, int i, int at) {
    return read_tile(wbuf(decltype(bc)::value, i / H) + wrow + 2048 * (i % H), at);
  };
  auto read_a = [&](auto bc, int j, int at) { return read_tile(abuf(decltype(bc)::value) + arow + 2048 * j, at); };
  auto read_s = [&](auto bc, int j) {
    return *reinterpret_cast<const float*>(sbuf(decltype(bc)::value) + 4 * (wm * 16 * J + 16 * j + l16));
  };

  v4f acc[2 * H][J];
  // MFMA results join their sums kLag slots later
  constexpr int kLag = kSlots % 4 == 0 ? 4 : kSlots % 3 == 0 ? 3 : 2;
  constexpr int kScales = kAhead && kGate ? 2 : 1;
  v4f pend[kLag];
  float c[kScales][J];  // the token tiles' scales for the products of a phase (of each half)
  // slot t of a phase takes token tile t / kG and weight tile wt(t), there and back, so that
  // every MFMA shares an operand with the one before it (4096 x 8192 -> 4096 114.7 -> 113.7 us)
  auto wt = [](int t) { return (t / kG) & 1 ? kG - 1 - t % kG : t % kG; };
  auto join = [&](int ph, int t) {  // the results of slot t of phase ph
    v4f& s = acc[kG * ph + wt(t)][t / kG];
    const float f = c[kScales == 2 ? wt(t) / H : 0][t / kG];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = __builtin_fmaf(pend[t % kLag][e], f, s[e]);
  };
  // slot t of phase ph: its MFMA; the results of the one kLag slots before it are added
  auto slot = [&](int ph, int t, const v8i& w, const v8i& a) {
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
    const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);  // (the MFMA first, the fmas beside it)
    if (t >= kLag) join(ph, t - kLag);
    else join((ph + kP - 1) % kP, kSlots + t - kLag);
    pend[t % kLag] = d;
  };
  static_assert(kSlots % kLag == 0, "the places of what is pending are those of the slots");

  using B0 = std::integral_constant<int, 0>;
  using B1 = std::integral_constant<int, 1>;
  using B2 = std::integral_constant<int, 2>;
  using B3 = std::integral_constant<int, 3>;
  int shift = 0;  // stages by which the DMAs run ahead into the next tile
  // stage q from buffer bc: its tokens, its token scales and the first phase's weights
  // are in registers
  auto iteration = [&](int q, auto bc) {
    constexpr int b = decltype(bc)::value, set = kAhead ? b & 1 : 0;
    using BC = std::integral_constant<int, b>;
    using BN = std::integral_constant<int, (b + 1) % R>;
    const float half = q == half_at ? 0.5f : 1.0f, up = kGate ? half * sw1 : 0.f;
    const float sw = half * sw0;
    float next[J];
#pragma unroll
    for (int ph = 0; ph < kP; ++ph) {
      if (ph == kP - 2) load_ws(q + 1);
      const bool last = ph == kP - 1, part = kTwice && ph == 1, after = kTwice && ph == 2;
      const Col col = stage_col(q + R + shift);
      const int at = at_row();
      if (last || part) {
        __builtin_amdgcn_sched_barrier(0);
        // this wave's reads of what is given back, and its DMAs of what is read next;
        // those issued after these may still be in flight
        wait_vm_lds<kTwice ? kDmas : (R - 2) * kDmas>();
        barrier();
        // (the last phase, which fetches what the next stage begins with, goes ahead of the
        // SIMD's other wave: 4096 x 8192 -> 4096 116 -> 115 us)
        if (kTwice && last) __builtin_amdgcn_s_setprio(1);
      }
      static_assert(kAhead || kP % 2 == 0, "the next stage's first phase takes the other weight registers");
      if (kAhead) load_ws(q + 1);
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        slot(ph, t, fw[kAhead ? set : ph & 1][wt(t)], fa[set][t / kG]);
        // (a token tile's scale is needed kLag slots after its first MFMA, and was kLag
        // slots after its last one)
        if ((ph == 0 || (kGate && ph == kP / 2)) && t % kG == kG - 1) {
          c[0][t / kG] = st[t / kG] * (ph == 0 ? sw : up);
          if constexpr (kScales == 2) c[1][t / kG] = st[t / kG] * up;
        }
        if (!last) {
          if (t < kG) fw[(ph + 1) & 1][t] = read_w(BC{}, kG * (ph + 1) + t, at);
        } else {
          if (t == 0) {
#pragma unroll
            for (int j = 0; j < J; ++j) next[j] = read_s(BN{}, j);
          }
          if constexpr (kAhead) {
            constexpr int kEach = (2 * H + J + kSlots - 1) / kSlots;  // fragments
#pragma unroll
            for (int f = kEach * t; f < kEach * (t + 1) && f < 2 * H + J; ++f) {
              if (f < J) fa[set ^ 1][f] = read_a(BN{}, f, at);
              else fw[set ^ 1][f - J] = read_w(BN{}, f - J, at);
            }
          } else {
            if (t < kG) fw[0][t] = read_w(BN{}, t, at);
            if (t % kG == kG - 1) fa[0][t / kG] = read_a(BN{}, t / kG, at);
          }
        }
        if (last || part || after) {  // the early DMAs are spread over two phases
          const int mid = (kEarly + 1) / 2;
          const int first = last && kTwice ? kEarly : after ? mid : 0, end = part ? mid : after ? kEarly : kDmas;
          const int each = (end - first + kSlots - 1) / kSlots;
#pragma unroll
          for (int k = first + each * t; k < first + each * (t + 1) && k < end; ++k) dma_one(k, col, BC{});
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (kTwice) __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int j = 0; j < J; ++j) st[j] = next[j];
  };
  int tile = blockIdx.x;
  dma_tile(tile);
  lane_offsets();
  dma_stage(0, B0{});
  dma_stage(1, B1{});
  if constexpr (R > 2) dma_stage(2, B2{});
  if constexpr (R > 3) dma_stage(3, B3{});
  wait_vm_lds<(R - 1) * kDmas + kLate>();
  barrier();
  for (;;) {
  const int tn0 = tn, nt = n0, mt = m0;  // of the products
  const size_t ws_at = (size_t)min((nt + wn * kWaveCols) >> 7, ((N + 127) >> 7) - 1) * S_all + q_begin;
  ws0 = (cfloat*)(p.g.w_scales + ws_at);
  ws1 = (cfloat*)((kGate ? p.g.up_scales : p.g.w_scales) + ws_at);
  load_ws(0);
#pragma unroll
  for (int t = 0; t < kG; ++t) fw[0][t] = read_w(B0{}, t, fo);
#pragma unroll
  for (int j = 0; j < J; ++j) fa[0][j] = read_a(B0{}, j, fo), st[j] = read_s(B0{}, j);
#pragma unroll
  for (int i = 0; i < 2 * H; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < kLag; ++t) pend[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < J; ++j) c[0][j] = c[kScales - 1][j] = 0.f;
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
  }
#pragma unroll
  for (int t = 0; t < kLag; ++t) join(kP - 1, kSlots + t - kLag);
  if constexpr (!kWhole) wait_vm_lds<0>();  // no DMA may land in a next workgroup's LDS

  if constexpr (kSplit) {
    // Every workgroup stores its fp32 sums with agent-coherent stores, waits for them and
    // bumps the tile's counter (which wraps to zero); the last to arrive adds all of them
    // in the order of K.
    constexpr int kWg = Sh::kWaves * 2 * H * J * 256;  // floats of a workgroup
    constexpr int kSc1 = 16;                           // cache policy: past the XCD's own L2
    const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
        p.part + (size_t)blockIdx.x * p.splits * kWg, 0, 4 * p.splits * kWg, 0x00027000);
    const int wave_at = 4 * wave * (2 * H * J * 256), lane_at = 16 * lane;
#pragma unroll
    for (int i = 0; i < 2 * H; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i][j]), part, lane_at + 1024 * (i * J + j),
                                               wave_at + 4 * kWg * (int)blockIdx.y, kSc1);
    __asm__ volatile("" ::: "memory");
    wait_vm_lds<0>();  // the partial is visible to the agent
    barrier();
    if (tid == 0) arrived = atomicInc(p.count + blockIdx.x, (u32)(p.splits - 1));
    __syncthreads();
    if (arrived != (u32)(p.splits - 1)) return;
    __asm__ volatile("" ::: "memory");
    // (the loads of as many splits as registers hold run together: 77 x 4096 -> 1536 on tiles of 64 x 64,
    // 4 / 8 / 16 splits, 8.6 / 10.5 / 15.2 us one by one, 8.4 / 9.4 / 12.7 together)
    auto add_splits = [&](int s, auto count) {
      constexpr int n = decltype(count)::value;
      v4u t[n][2 * H][J];
#pragma unroll
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int i = 0; i < 2 * H; ++i)
#pragma unroll
          for (int j = 0; j < J; ++j)
            t[k][i][j] =
                __builtin_amdgcn_raw_buffer_load_b128(part, lane_at + 1024 * (i * J + j), wave_at + 4 * kWg * (s + k), kSc1);
#pragma unroll
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int i = 0; i < 2 * H; ++i)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const v4f v = __builtin_bit_cast(v4f, t[k][i][j]);
            acc[i][j] = k == 0 && s == 0 ? v : acc[i][j] + v;
          }
    };
    constexpr int kTogether = std::max(1, std::min(8, 16 / (H * J)));  // a power of two, as the splits are
    using Together = std::integral_constant<int, kTogether>;
    using Half = std::integral_constant<int, std::max(1, kTogether / 2)>;
    using Quarter = std::integral_constant<int, std::max(1, kTogether / 4)>;
    if (p.splits >= Together::value)
      for (int s = 0; s < p.splits; s += Together::value) add_splits(s, Together{});
    else if (p.splits >= Half::value) add_splits(0, Half{});
    else add_splits(0, Quarter{});
  }

  // The epilogue, in fp32 from the sums.  A wave turns its tile 16 token rows at a time
  // through LDS of its own, so that rows leave in runs of 16 bytes per lane.
  int el = lane;
  __asm__ volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(el));
  const int e16 = el & 15, eq = el >> 4;
  uint8_t* turn = rows + wave * Sh::kTurn;
  const int nw = nt + wn * kWaveCols, mw = mt + wm * 16 * J;  // the wave's first column and row
  auto bias4 = [&](const uint16_t* b, int n, float (&f)[4]) {
    const uint2 v = b != nullptr ? *reinterpret_cast<const uint2*>(b + min(n, N - 4)) : uint2{0u, 0u};
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  };
  if constexpr (kGate) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int n = nw + 16 * i + 4 * eq;
      float bg[4], bu[4];
      bias4(p.g.bias, n, bg);
      bias4(p.g.up_bias, n, bu);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = gate_act(acc[i][j][e] + bg[e], p.g.epilogue) * (acc[H + i][j][e] + bu[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) {
      float b[4];
      bias4(p.g.bias, nw + 16 * i + 4 * eq, b);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float o = acc[i][j][e] + b[e];
          acc[i][j][e] = p.g.epilogue == kEpilogueGelu ? gelu_exp2(o) : o;
        }
    }
  }
  if constexpr (kForm == kGatedCodes) {
    // a token's block of 128 features lies in the WN waves of a tile row: their
    // maxima meet in LDS.  Features past the end (a half last block) are whole waves'
    static_assert(kCols == 128, "a tile holds a block of features");
    const bool in = kWhole || nw < N;
    if (p.g.smooth != nullptr) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float4 s = *reinterpret_cast<const float4*>(p.g.smooth + min(nw + 16 * i + 4 * eq, N - 4));
        const float mu[4] = {1.0f / s.x, 1.0f / s.y, 1.0f / s.z, 1.0f / s.w};
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] *= mu[e];
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < H; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = BitMaxOp::run(m, __builtin_fabsf(acc[i][j][e]));
      m = max_rows4(in ? m : 0.f);
      if (eq == 0) red[(wn * WM + wm) * 16 * J + 16 * j + e16] = m;
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's maxima are in LDS
    barrier();
    if (!in) return;  // (of the one tile: whole ones have all features)
    constexpr int kRow = 16 * H;  // bytes of a row of the wave's codes
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float m = red[wm * 16 * J + 16 * j + e16];
#pragma unroll
      for (int w = 1; w < WN; ++w) m = BitMaxOp::run(m, red[(w * WM + wm) * 16 * J + 16 * j + e16]);
      float s, inv;
      block_scale(m, s, inv);
      const int tok = mw + 16 * j + e16;
      if (wn == 0 && eq == 0 && tok < M) p.g.out_scales[(size_t)tn0 * p.g.out_stride + tok] = s;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        const u32 q4 = fp8_codes4(v, inv);
        *reinterpret_cast<u32*>(turn + e16 * kRow + 16 * (i ^ ((e16 >> 1) & (H - 1))) + 4 * eq) = inv == 0.f ? 0u : q4;
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes are done
      __asm__ volatile("" ::: "memory");
      const int ml = el / H, ch = el - ml * H;
      const int m2 = mw + 16 * j + ml;
      if (el < 16 * H) {
        const v4u v = *reinterpret_cast<const v4u*>(turn + ml * kRow + 16 * (ch ^ ((ml >> 1) & (H - 1))));
        if (m2 < M) *reinterpret_cast<v4u*>(static_cast<uint8_t*>(p.g.out) + (size_t)m2 * N + nw + 16 * ch) = v;
      }
      __asm__ volatile("" ::: "memory");  // (a wave's LDS operations run in order)
    }
  } else {
    // bf16 rows, 16 H columns of a half at a time
    constexpr int kChunks = 2 * H, kMask = kChunks - 1;  // 16-byte chunk c of row m sits at c ^ (m & kMask)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int h = 0; h < (kGate ? 1 : 2); ++h) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const v4f& o = acc[h * H + i][j];
          const int nl = 16 * i + 4 * eq;
          uint8_t* dst = turn + e16 * (16 * kChunks) + (((nl >> 3) ^ (e16 & kMask)) << 4) + 8 * (eq & 1);
          *reinterpret_cast<uint2*>(dst) = uint2{pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3])};
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes are done
        __asm__ volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < (H + 1) / 2; ++t) {
          const int at = 64 * t + el;
          const int ml = at / kChunks, ch = at - ml * kChunks;
          const int m = mw + 16 * j + ml, n = nw + h * 16 * H + 8 * ch;
          if (at < 16 * kChunks) {
            const v4u v = *reinterpret_cast<const v4u*>(turn + ml * (16 * kChunks) + ((ch ^ (ml & kMask)) << 4));
            // N % 64 == 0, so n < N covers n + 7
            if (m < M && n < N)
              __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(static_cast<uint16_t*>(p.g.out) + (size_t)m * N + n));
          }
        }
        __asm__ volatile("" ::: "memory");  // (a wave's LDS operations run in order)
      }
  }
  if (!more) break;
  tile = next;
  }
  if constexpr (kWhole) wait_vm_lds<0>();  // no DMA may land in a next workgroup's LDS
}

struct Plan {
  int shape;    // index into kShapes
  int tiles;
  int splits;
  double cost;  // us, by the model below
};

// Workgroup tiles, the test hook's name of each (weight rows / 64, tokens / 64, LDS stages)
// and what a launch takes by the model of w8a8_gemm.hip: base + n (fill + S step) us with n
// workgroups on the busiest compute unit and S stages of 128 k, pairs of workgroups at fill2
// and step2 where two share a compute unit.  Fitted to picks, not to times: to 554 shapes (17
// to 4608 tokens, K 512 to 10240, 384 to 12288 rows, 40 % of them gated), times far from a
// shape's best weighing less.  On 2373 other shapes (profiles/plan_sweep_fp8.txt) what a
// call takes is 0.2 % from the best tile and split on the geometric mean, 29 % at most (817 x 9344 ->
// 2816: 432 in 4 splits 51.6 us, 224 whole 40.0).  The times that it gives are 7 % low on the mean,
// 13 % (up to 23) for 4096 and more tokens with K from 8192, where power lowers the clock:
// a round of 442 takes 1.65 us a stage there, not 1.302.  Its picks are as near the best there: 2.7 %
// below the best single launch on the mean, 26 % above at most (4150 x 15360 -> 576: 442 in 4 splits 73.5 us, 224 whole 58.2).
#define SVDQ_SHAPES(X)                                   \
  X(442, 4, 4, 2, 4, 2, -5.64, 13.89, 1.302, 0.0, 0.0)   \
  X(432, 4, 3, 2, 4, 2, -2.69, 9.82, 1.035, 0.0, 0.0)    \
  X(423, 2, 4, 4, 2, 3, -0.37, 6.26, 0.863, 0.0, 0.0)    \
  X(413, 2, 2, 4, 2, 3, 0.83, 3.53, 0.647, 0.0, 0.0)     \
  X(224, 2, 2, 2, 4, 4, 0.78, 3.91, 0.517, 0.0, 0.0)     \
  X(213, 2, 2, 2, 2, 3, 3.24, 0.44, 0.381, 2.02, 0.703)  \
  X(114, 1, 2, 2, 2, 4, 2.52, 1.10, 0.248, 1.79, 0.488)
struct ShapeInfo {
  int code, tn, tm, waves, wgs;
  double base, fill, step, fill2, step2;
};
template <int H, int J, int WN, int WM, int R>
constexpr ShapeInfo info(int code, double base, double fill, double step, double fill2, double step2) {
  using S = Shape<H, J, WN, WM, R>;
  return ShapeInfo{code, S::kTN, S::kTM, S::kWaves, S::kWgs, base, fill, step, fill2, step2};
}
#define SVDQ_INFO(code, h, j, wn, wm, r, base, fill, step, fill2, step2) \
  info<h, j, wn, wm, r>(code, base, fill, step, fill2, step2),
constexpr ShapeInfo kShapes[] = {SVDQ_SHAPES(SVDQ_INFO)};
#undef SVDQ_INFO
constexpr int kMaxSplits = 16;

std::atomic<int> g_tile{0}, g_splits{0};  // test hook

Form form_of(const Fp8Args& a) { return a.up == nullptr ? kPlain : a.out_scales == nullptr ? kGated : kGatedCodes; }

int64_t tiles_of(const ShapeInfo& s, const Fp8Args& a) {
  const int64_t cols = a.up != nullptr ? s.tn / 2 : s.tn;
  return ((a.N + cols - 1) / cols) * (((int64_t)a.M + s.tm - 1) / s.tm);
}

// the cheapest tile and K-split
Plan plan_of(const Fp8Args& a) {
  const int cus = current_cus();
  const int stages = (a.K + 127) / 128;
  const Form form = form_of(a);
  const int forced_tile = g_tile.load(std::memory_order_relaxed), forced = g_splits.load(std::memory_order_relaxed);
  Plan best{-1, 0, 1, 0.0};
  for (int i = 0; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i) {
    const ShapeInfo& s = kShapes[i];
    if (form == kGatedCodes && s.tn != 256) continue;  // a tile holds a block of features
    if (forced_tile > 1 && forced_tile != s.code && !(form == kGatedCodes && forced_tile / 100 != 4)) continue;
    const int64_t tiles = tiles_of(s, a);
    if (tiles * s.waves * 64 >= (1ll << 32)) continue;  // a launch holds fewer than 2^32 threads
    for (int splits = 1; splits <= std::min(kMaxSplits, stages); splits *= 2) {
      const int64_t wgs = tiles * splits;
      if (splits > 1 && tiles > (int64_t)kWsMaxCounters) break;
      if (forced > 0 ? splits > forced : splits > 1 && wgs > 2 * cus) break;
      const double n = (double)((wgs + cus - 1) / cus), S = (double)((stages + splits - 1) / splits);
      double cost = s.base;
      if (s.wgs == 2) {
        const double pairs = std::floor(n / 2);
        cost += pairs * (s.fill2 + S * s.step2) + (n - 2 * pairs) * (s.fill + S * s.step);
      } else {
        cost += n * (s.fill + S * s.step);
      }
      if (splits > 1) cost += -0.56 + 0.70 * splits + 0.88 * (s.tn / 64) * (s.tm / 64);  // the partials' round trips
      if (best.shape < 0 || cost < best.cost || (forced > 0 && best.shape == i)) best = Plan{i, (int)tiles, splits, cost};
    }
  }
  return best;
}

// The launches of a product: the tokens [0, m1) in whole rounds of one of the largest
// tiles, and the rest on the tile that suits it (m1 = M: one launch).  The last round of a
// large tile otherwise leaves most compute units idle.
// kSecondLaunch: what a second launch takes beyond the model's sum, in us.
constexpr double kSecondLaunch = 6.5;
struct Launches {
  int64_t m1;
  Plan first, rest;
};
Fp8Args part_of(const Fp8Args& a, int64_t m0, int64_t m1) {
  Fp8Args part = a;
  part.M = (int)(m1 - m0);
  part.act += (size_t)m0 * (size_t)a.K;
  part.act_scales += m0;
  part.out = static_cast<uint8_t*>(a.out) + (size_t)m0 * (size_t)a.N * (a.out_scales != nullptr ? 1 : 2);
  if (a.out_scales != nullptr) part.out_scales += m0;
  return part;
}
Launches plan_launches(const Fp8Args& a, bool forced, int cus) {
  Launches best{a.M, plan_of(a), Plan{}};
  if (forced) return best;
  const double S = (double)((a.K + 127) / 128);
  double best_cost = best.first.cost;
  for (int i = 0; i < 3; ++i) {
    const ShapeInfo& s = kShapes[i];
    const int64_t cols = a.up != nullptr ? s.tn / 2 : s.tn;
    const int64_t nt = (a.N + cols - 1) / cols, mt = (a.M + s.tm - 1) / s.tm;
    const int64_t rounds = nt * mt / cus, mt1 = rounds * cus / nt;
    if (mt1 <= 0 || mt1 * s.tm >= a.M || mt1 * nt * s.waves * 64 >= (1ll << 32)) continue;
    Fp8Args rest = a;
    rest.M = (int)(a.M - mt1 * s.tm);
    Launches l{mt1 * s.tm, Plan{i, (int)(mt1 * nt), 1, 0.0}, plan_of(rest)};
    l.first.cost = kSecondLaunch + s.base + (double)((mt1 * nt + cus - 1) / cus) * (s.fill + S * s.step);
    if (l.first.cost + l.rest.cost < best_cost) {
      best = l;
      best_cost = l.first.cost + l.rest.cost;
    }
  }
  return best;
}

// Planned once for a call's workspace query, its check and its launch: a thread keeps its
// last plan, by all that it depends on (up to 1 us each time otherwise).
Launches launches_of(const Fp8Args& a) {
  struct Last {
    std::array<int, 7> key;
    Launches plan;
  };
  thread_local Last last{};
  const int tile = g_tile.load(std::memory_order_relaxed), splits = g_splits.load(std::memory_order_relaxed);
  const int cus = current_cus();
  const std::array<int, 7> key{a.M, a.N, a.K, (int)form_of(a), tile, splits, cus};
  if (last.key != key) last = Last{key, plan_launches(a, tile > 1 || splits > 0, cus)};
  return last.plan;
}

template <int H, int J, int WN, int WM, int R, Form kForm>
void tile_form(const TileArgs& t, int tiles, hipStream_t stream) {
  using Sh = Shape<H, J, WN, WM, R>;
  const dim3 block(Sh::kThreads);
  // whole tiles, more than the chip holds at once, and no long K: one workgroup per compute
  // unit (of the largest tile, which the plan takes for such products).  Four rounds of
  // 256 x 256: K 2304 153.6 -> 149.5 us, 3072 187.2 -> 185.6, 8192 446.5 -> 450.7
  if constexpr (H == 4) {
    const int cus = current_cus();
    if (t.splits == 1 && tiles > cus && t.g.M % Sh::kTM == 0 && t.g.N % (kForm == kPlain ? Sh::kTN : Sh::kTN / 2) == 0 &&
        (t.g.K + 127) / 128 % R == 0 && t.g.K <= 4096) {
      hipLaunchKernelGGL((fp8_tile_kernel<H, J, WN, WM, R, kForm, kMany>), dim3(cus), block, 0, stream, t);
      return;
    }
  }
  if (t.splits > 1)
    hipLaunchKernelGGL((fp8_tile_kernel<H, J, WN, WM, R, kForm, kSplits>), dim3(tiles, t.splits), block, 0, stream, t);
  else
    hipLaunchKernelGGL((fp8_tile_kernel<H, J, WN, WM, R, kForm, kOne>), dim3(tiles), block, 0, stream, t);
}

template <int H, int J, int WN, int WM, int R>
hipError_t tile_go(const TileArgs& t, int tiles, hipStream_t stream) {
  switch (form_of(t.g)) {
    case kPlain: tile_form<H, J, WN, WM, R, kPlain>(t, tiles, stream); break;
    case kGated: tile_form<H, J, WN, WM, R, kGated>(t, tiles, stream); break;
    case kGatedCodes:
      if constexpr (Shape<H, J, WN, WM, R>::kTN == 256) tile_form<H, J, WN, WM, R, kGatedCodes>(t, tiles, stream);
      else return hipErrorInvalidValue;
      break;
  }
  return hipGetLastError();
}

// The weight-streaming kernel for up to 16 tokens, but where K is long beside its N / 16
// workgroups, which do not divide K among themselves, or the rows are many.  Measured, it
// against the best tile and split, weights from HBM, us, 1 / 4 / 16 tokens
// (profiles/few_token_rule_fp8.txt):
//   plain  4096 -> 2048   5.2 / 5.6* / 6.4*       against  8.2 / 8.3 / 8.3
//          4096 -> 16384  14.9 / 15.4* / 20.3     against  17.4 / 17.5 / 17.5*
//          8192 -> 64     6.4 / 7.0* / 9.0        against  7.5 / 7.5 / 7.5*
//         16384 -> 64     10.7 / 12.0 / 16.0      against  8.8 / 8.7* / 8.8*
//         16384 -> 4096   15.9 / 16.6* / 21.3     against  18.6 / 18.8 / 19.2*
//         65536 -> 64     36.9 / 42.4 / 57.9      against  14.2 / 14.0* / 14.0*
//   gated  4096 -> 2048   7.8 / 7.9* / 8.9*       against  9.3 / 9.4 / 9.4
//          8192 -> 1024   11.6 / 12.4 / 14.6      against  9.9 / 9.9* / 10.1*
//          8192 -> 4096   16.2 / 16.6* / 18.4     against  17.4 / 17.9 / 17.9*
//         16384 -> 8192   49.1 / 49.7* / 56.9     against  46.7 / 50.8 / 51.3*
//         65536 -> 64     67.1 / 72.6 / 90.6      against  14.8 / 14.8* / 14.9*
//   codes  8192 -> 64     11.2 / 11.7* / 14.0*    against  14.4 / 14.4 / 14.5
//         16384 -> 64     19.0 / 20.2* / 24.3     against  17.6 / 17.7 / 17.8*
//         16384 -> 1024   21.0 / 22.2* / 26.7     against  22.8 / 22.9 / 23.3*
//         65536 -> 64     66.3 / 72.2 / 89.2      against  31.4 / 31.5* / 31.6*
// (* marks the side the rule takes, up to 4 and up to 16 tokens.)
bool few_tokens(const Fp8Args& a) {
  const int t = g_tile.load(std::memory_order_relaxed);
  if (t > 1 || a.M > 16) return false;
  if (t == 1) return true;
  const bool gated = a.up != nullptr;
  if (a.out_scales != nullptr) return a.K <= (a.M <= 4 ? 16384 : 8192);
  if (a.K > (gated ? 4096 : 8192)) return a.M <= 4 && a.N >= 4096;  // a workgroup for each compute unit
  if (a.K > 4096) return a.M <= 4;
  return a.M <= 4 || (gated ? 2 : 1) * (int64_t)a.N <= 8192;
}

size_t plan_bytes(const Plan& p) {
  if (p.splits <= 1) return 0;
  const ShapeInfo& s = kShapes[p.shape];
  return ws_bytes((size_t)p.tiles, (size_t)p.tiles * p.splits * s.tn * s.tm * sizeof(float));
}

}  // namespace

bool fp8_tile_known(int tile) {
  if (tile == 0 || tile == 1) return true;
  for (const ShapeInfo& s : kShapes)
    if (s.code == tile) return true;
  return false;
}

void set_fp8_plan_override(int tile, int splits) {
  g_tile.store(tile, std::memory_order_relaxed);
  g_splits.store(splits, std::memory_order_relaxed);
}

size_t fp8_workspace_bytes(const Fp8Args& a) {
  if (few_tokens(a)) return fp8_skinny_workspace_bytes(a);
  const Launches l = launches_of(a);
  return std::max(plan_bytes(l.first), l.m1 < a.M ? plan_bytes(l.rest) : 0);
}

static hipError_t launch_plan(const Fp8Args& a, const Plan& p, const Workspace& ws, hipStream_t stream) {
  if (p.shape < 0 || plan_bytes(p) > ws.bytes) return hipErrorInvalidValue;
  TileArgs t{a, p.splits, p.tiles, nullptr, nullptr};
  if (p.splits > 1) {
    t.count = ws_counters(ws);
    t.part = static_cast<float*>(ws_scratch(ws));
  }
  switch (kShapes[p.shape].code) {
#define SVDQ_GO(code, h, j, wn, wm, r, base, fill, step, fill2, step2) \
  case code: return tile_go<h, j, wn, wm, r>(t, p.tiles, stream);
    SVDQ_SHAPES(SVDQ_GO)
#undef SVDQ_GO
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_fp8_gemm(const Fp8Args& a, Workspace ws, hipStream_t stream) {
  if (few_tokens(a)) return launch_fp8_skinny(a, ws, stream);
  const Launches l = launches_of(a);
  const hipError_t e = launch_plan(part_of(a, 0, l.m1), l.first, ws, stream);
  if (e != hipSuccess || l.m1 == a.M) return e;
  return launch_plan(part_of(a, l.m1, a.M), l.rest, ws, stream);
}

}  // namespace svdq
