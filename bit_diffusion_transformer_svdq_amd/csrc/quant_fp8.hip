// The block quantizer of the 8-bit floating-point linear (gfx950):
//   x_hat = x, or bf16(fl32(x fl32(1/smooth)))
//   s = fl32(max|x_hat| fl32(1/448)) over a row's 128 channels, q = e4m3(fl32(x_hat fl32(1/s)))
//
// Bound by HBM: x is read once (2 bytes) and the codes are written once.  A lane
// holds 8 channels of a row, so a block of 128 is one DPP row of 16 lanes and its
// maximum takes four rotations: no LDS, no barrier.  A wave takes kRows rows of the
// same 512 channels: all their loads are in flight together, the smoothing
// reciprocals are taken once, and lane r keeps row r's scale, so that scales (one row
// per block, as the product reads them) leave as runs of kRows floats.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8.h"

namespace svdq {
namespace {

constexpr int kWaves = 4;

template <int kRows, bool kSmooth>
__global__ __launch_bounds__(64 * kWaves) void quant_fp8_kernel(const QuantFp8Args a, int col_groups) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  // (column groups of a row run are neighbours: they share its lines of x)
  const int64_t run = wave / col_groups;
  const int cg = (int)(wave - run * col_groups);
  const int64_t row0 = run * kRows;
  if (row0 >= a.M) return;
  const int rows = (int)min((int64_t)kRows, a.M - row0);
  const int c = 512 * cg + 8 * lane;
  const bool live = c < a.K;             // K % 64 == 0: 8 channels are in or out together
  const int cc = live ? c : a.K - 8;

  uint4 p[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    p[r] = *reinterpret_cast<const uint4*>(a.x + (size_t)(row0 + min(r, rows - 1)) * a.K + cc);
  float mu[8];
  if constexpr (kSmooth) {
    const float4 s0 = *reinterpret_cast<const float4*>(a.smooth + cc);
    const float4 s1 = *reinterpret_cast<const float4*>(a.smooth + cc + 4);
    mu[0] = s0.x, mu[1] = s0.y, mu[2] = s0.z, mu[3] = s0.w, mu[4] = s1.x, mu[5] = s1.y, mu[6] = s1.z, mu[7] = s1.w;
    recip8(mu);
  }
  float keep = 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float f[8];
    unpack8(p[r], f);
    if constexpr (kSmooth) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= mu[e];
      unpack8(pack8(f), f);
    }
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = BitMaxOp::run(amax, __builtin_fabsf(f[e]));
    if (!live) amax = 0.f;  // the half of a last block that is not there
    amax = max16(amax);
    float s, inv;
    block_scale(amax, s, inv);
    if ((lane & 15) == r) keep = s;
    row_v2u q = {fp8_codes4(&f[0], inv), fp8_codes4(&f[4], inv)};
    if (inv == 0.f) q = row_v2u{0u, 0u};
    if (live && r < rows) *reinterpret_cast<row_v2u*>(a.codes + (size_t)(row0 + r) * a.K + c) = q;
  }
  const int block = 4 * cg + (lane >> 4);
  if (kFp8Block * block < a.K && (lane & 15) < rows)
    a.scales[(size_t)block * a.scale_stride + row0 + (lane & 15)] = keep;
}

template <int kRows>
hipError_t go(const QuantFp8Args& a, hipStream_t stream) {
  const int col_groups = (a.K + 511) / 512;
  const int64_t waves = (int64_t)((a.M + kRows - 1) / kRows) * col_groups;
  const int64_t wgs = (waves + kWaves - 1) / kWaves;
  if (wgs * 64 * kWaves >= (1ll << 32)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)wgs), block(64 * kWaves);
  if (a.smooth != nullptr) hipLaunchKernelGGL((quant_fp8_kernel<kRows, true>), grid, block, 0, stream, a, col_groups);
  else hipLaunchKernelGGL((quant_fp8_kernel<kRows, false>), grid, block, 0, stream, a, col_groups);
  return hipGetLastError();
}

}  // namespace

// Rows per wave: one while a compute unit has no more than 64 waves of one row, else four
// (us, x from HBM, 1 / 2 / 4 / 8 / 16 rows: 512 x 3840 3.5 / 3.9 / 4.2 / 5.2 / 7.4; 1333 x 1920 3.9 / 4.4 /
// 4.8 / 5.3 / 7.6, smoothed 4.8 / 4.9 / 5.6 / 6.2 / 8.8; 4608 x 3072 11.2 / 11.6 / 10.4 / 11.4 / 12.8, smoothed
// 13.7 / 12.8 / 11.9 / 13.2 / 14.7: 4.1 TB/s, 3.6 smoothed).
// 2^24 rows of 65536 channels would be 2^29 waves, past the launch limit of 2^32
// threads: such calls are cut into parts of whole runs.
hipError_t launch_quant_fp8(const QuantFp8Args& args, hipStream_t stream) {
  QuantFp8Args a = args;
  const int64_t col_groups = (a.K + 511) / 512;
  const bool one = args.M * col_groups <= 64 * (int64_t)current_cus();
  const int64_t most = ((1ll << 25) / col_groups) * 4;  // rows whose waves stay below 2^25
  for (int64_t m = 0; m < args.M; m += most) {
    a.M = (int)std::min<int64_t>(most, args.M - m);
    a.x = args.x + (size_t)m * args.K;
    a.codes = args.codes + (size_t)m * args.K;
    a.scales = args.scales + m;
    const hipError_t e = one ? go<1>(a, stream) : go<4>(a, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace svdq
