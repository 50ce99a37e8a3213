// The 8-bit floating-point linear for up to 16 tokens on gfx950, plain and gated: a
// weight stream.
//
// With few tokens the product is bound by reading the weights once (N K bytes, twice
// that gated).  A workgroup owns 16 weight rows (gated: 16 rows of each projection) and
// its 4 or 8 waves divide the blocks of K: each wave reads its part of the rows straight into
// registers (16 rows x 128 bytes, the K of one v_mfma_f32_16x16x128_f8f6f4, in two load
// instructions), the same part of the token rows from L2, and adds each block's product to
// fp32 sums with the block's scale.  The waves' sums are added in LDS in wave order.
//
// Codes as output need the largest of a token's 128 features, those of 8 workgroups:
// each leaves its H as fp32 in the workspace, and the last of the eight to arrive
// quantizes the block.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"

namespace svdq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBatch = 2;  // blocks loaded together
constexpr int kMaxTokens = 16;

struct SkinnyArgs {
  Fp8Args g;
  row_u32* count;  // one arrival counter per block of features (coded output)
  float* h;        // fp32 [N / 16][16 tokens][16 features]
};

template <int kWaves, bool kGate, bool kCodes>
__global__ __launch_bounds__(64 * kWaves) void fp8_skinny_kernel(const SkinnyArgs p) {
  constexpr int kProj = kGate ? 2 : 1;
  __shared__ __attribute__((aligned(16))) v4f red[kWaves][kProj][64];
  __shared__ row_u32 arrived;
  const Fp8Args& a = p.g;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int KB = (a.K + 127) >> 7;
  const int b0 = (int)((long)wave * KB / kWaves), b1 = (int)((long)(wave + 1) * KB / kWaves);

  // lane (l16, lq) takes bytes 16 lq .. and 64 + 16 lq .. of a block of row l16
  const size_t wo = (size_t)(n0 + l16) * a.K + 16 * lq;  // N % 64 == 0
  const uint8_t* wr[kProj];
  const float* sw[kProj];
  wr[0] = a.w + wo;
  sw[0] = a.w_scales + (size_t)(n0 >> 7) * KB;
  if constexpr (kGate) {
    wr[1] = a.up + wo;
    sw[1] = a.up_scales + (size_t)(n0 >> 7) * KB;
  }
  const int tok = min(l16, a.M - 1);
  const uint8_t* ar = a.act + (size_t)tok * a.K + 16 * lq;
  const float* sx = a.act_scales + tok;
  v4f acc[kProj];
#pragma unroll
  for (int j = 0; j < kProj; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};

  struct Batch {
    v4i w[kBatch][kProj][2], a[kBatch][2];
    float sx[kBatch], sw[kBatch][kProj];
  };
  // blocks past the wave's range repeat its last one (their products are not
  // added), so every load of a batch is unconditional; the missing half of a last
  // block of 64 repeats the first in both operands, and its scale is halved
  auto fetch = [&](Batch& f, int b) {
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int at = min(b + s, b1 - 1);
      const int off = 128 * at, hi = off + 64 < a.K ? off + 64 : off;
#pragma unroll
      for (int j = 0; j < kProj; ++j) {
        f.w[s][j][0] = *reinterpret_cast<const v4i*>(wr[j] + off);
        f.w[s][j][1] = *reinterpret_cast<const v4i*>(wr[j] + hi);
        f.sw[s][j] = sw[j][at];
      }
      f.a[s][0] = *reinterpret_cast<const v4i*>(ar + off);
      f.a[s][1] = *reinterpret_cast<const v4i*>(ar + hi);
      f.sx[s] = sx[(size_t)at * a.act_stride];
    }
  };
  auto add = [&](const Batch& f, int b) {
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (b + s < b1) {
        const float twice = 128 * (b + s) + 64 >= a.K ? 0.5f : 1.0f;
        const v4i x0 = f.a[s][0], x1 = f.a[s][1];
        const v8i xa = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
#pragma unroll
        for (int j = 0; j < kProj; ++j) {
          const v4i y0 = f.w[s][j][0], y1 = f.w[s][j][1];
          const v8i wa = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
          const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xa, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
          const float c = f.sx[s] * (twice * f.sw[s][j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(d[e], c, acc[j][e]);
        }
      }
  };
  if (b0 < b1) {  // K may have fewer blocks than the workgroup waves
    Batch f0, f1;
    fetch(f0, b0);
    int b = b0;
    for (; b + 2 * kBatch < b1; b += 2 * kBatch) {
      fetch(f1, b + kBatch);
      add(f0, b);
      fetch(f0, b + 2 * kBatch);
      add(f1, b + kBatch);
    }
    if (b + kBatch < b1) {
      fetch(f1, b + kBatch);
      add(f0, b);
      add(f1, b + kBatch);
    } else {
      add(f0, b);
    }
  }
#pragma unroll
  for (int j = 0; j < kProj; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  const int m = l16, n = n0 + 4 * lq;  // the lane's token and first of four channels
  if (wave == 0) {
    v4f s[kProj];
#pragma unroll
    for (int j = 0; j < kProj; ++j) {
      s[j] = red[0][j][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s[j] += red[w][j][lane];
      const uint16_t* bias = j == 0 ? a.bias : a.up_bias;
      if (bias != nullptr) {
        const uint2 b2 = *reinterpret_cast<const uint2*>(bias + n);
        s[j] += v4f{bf16_lo(b2.x), bf16_hi(b2.x), bf16_lo(b2.y), bf16_hi(b2.y)};
      }
    }
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kGate) o[e] = gate_act(s[0][e], a.epilogue) * s[kProj - 1][e];
      else o[e] = a.epilogue == kEpilogueGelu ? gelu_exp2(s[0][e]) : s[0][e];
    }
    if constexpr (!kCodes) {
      if (m < a.M)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (size_t)m * a.N + n) =
            uint2{pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3])};
    } else {
      typedef unsigned long long u64;
      typedef float v2f __attribute__((ext_vector_type(2)));
      if (a.smooth != nullptr) {
        const float4 sm = *reinterpret_cast<const float4*>(a.smooth + n);
        o[0] *= 1.0f / sm.x, o[1] *= 1.0f / sm.y, o[2] *= 1.0f / sm.z, o[3] *= 1.0f / sm.w;
      }
      u64* h = reinterpret_cast<u64*>(p.h + (size_t)blockIdx.x * 256 + 16 * l16 + 4 * lq);
      __hip_atomic_store(h, __builtin_bit_cast(u64, v2f{o[0], o[1]}), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(h + 1, __builtin_bit_cast(u64, v2f{o[2], o[3]}), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __asm__ volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): H is visible to the agent
      __asm__ volatile("" ::: "memory");
      const int of = min(8, (a.N >> 4) - (int)(blockIdx.x & ~7u));  // workgroups of this block
      if (lane == 0) arrived = atomicInc(p.count + (blockIdx.x >> 3), (row_u32)(of - 1)) == (row_u32)(of - 1);
    }
  }
  if constexpr (kCodes) {
    typedef unsigned long long u64;
    typedef float v2f __attribute__((ext_vector_type(2)));
    __syncthreads();
    if (arrived == 0) return;
    __asm__ volatile("" ::: "memory");
    // 16 lanes per token, 8 features each; 4 tokens per wave
    const int t = 4 * wave + (lane >> 4), f = 8 * l16;
    if (wave >= (a.M + 3) / 4) return;
    const int blk = blockIdx.x & ~7u;
    const bool in = 16 * blk + f < a.N;  // a last block may hold 64 features
    const u64* h = reinterpret_cast<const u64*>(p.h + (size_t)(blk + (in ? f >> 4 : 0)) * 256 + 16 * t + (f & 15));
    float v[8];
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const v2f x = __builtin_bit_cast(v2f, __hip_atomic_load(h + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
      v[2 * e] = x[0], v[2 * e + 1] = x[1];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = BitMaxOp::run(amax, __builtin_fabsf(v[e]));
    amax = max16(in ? amax : 0.f);
    float s, inv;
    block_scale(amax, s, inv);
    row_v2u q = {fp8_codes4(&v[0], inv), fp8_codes4(&v[4], inv)};
    if (inv == 0.f) q = row_v2u{0u, 0u};
    if (t >= a.M) return;
    if (in) *reinterpret_cast<row_v2u*>(static_cast<uint8_t*>(a.out) + (size_t)t * a.N + 16 * blk + f) = q;
    if (l16 == 0) a.out_scales[(size_t)(blockIdx.x >> 3) * a.out_stride + t] = s;
  }
}

}  // namespace

// Waves per workgroup: four up to 16 blocks of K (each wave then has a batch or two) and
// into codes, else eight.  Measured, one token, weights from HBM, 4 / 8 waves, us: K 1024 -> 9216 4.2 / 5.9,
// gated 6.7 / 9.8, into codes 8.8 / 12.3; 1536 -> 1536 3.2 / 3.6, 4.1 / 4.8, 6.2 / 6.9; 2304 -> 6144 6.2 /
// 5.7, 9.9 / 9.3, 11.4 / 11.0; 3072 -> 12288 11.1 / 10.2, 17.6 / 17.7, 19.3 / 22.1; 12288 -> 3072 15.4 / 13.4,
// 20.8 / 21.5, 22.2 / 22.6.  (16 waves, and batches of one and four blocks, were no better: 3072 -> 12288
// 13.6, 10.5, 11.9.)  10.2 us is 3.7 TB/s over the weights, launch included.
size_t fp8_skinny_workspace_bytes(const Fp8Args& a) {
  if (a.out_scales == nullptr) return 0;
  return ws_bytes((size_t)(a.N + 127) / 128, (size_t)a.N * kMaxTokens * sizeof(float));
}

hipError_t launch_fp8_skinny(const Fp8Args& a, Workspace ws, hipStream_t stream) {
  if (a.M > kMaxTokens || fp8_skinny_workspace_bytes(a) > ws.bytes) return hipErrorInvalidValue;
  SkinnyArgs p{a, nullptr, nullptr};
  const dim3 grid(a.N / 16);
  const bool four = a.K <= 2048;
  if (a.up == nullptr) {
    if (four) hipLaunchKernelGGL((fp8_skinny_kernel<4, false, false>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((fp8_skinny_kernel<8, false, false>), grid, dim3(512), 0, stream, p);
  } else if (a.out_scales == nullptr) {
    if (four) hipLaunchKernelGGL((fp8_skinny_kernel<4, true, false>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((fp8_skinny_kernel<8, true, false>), grid, dim3(512), 0, stream, p);
  } else {
    p.count = ws_counters(ws);
    p.h = static_cast<float*>(ws_scratch(ws));
    hipLaunchKernelGGL((fp8_skinny_kernel<4, true, true>), grid, dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace svdq
