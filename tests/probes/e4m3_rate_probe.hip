// What MI355X (gfx950) reaches on e4m3 matrix instructions fed from registers, alone and
// with the fmas that a scale per block of K takes.  Not part of the library or the tests:
// a measurement program whose printed figures back the rates that the 8-bit
// floating-point linear is held against.
//
//   hipcc --offload-arch=gfx950 -O3 -std=c++17 -Xclang -target-feature
//         -Xclang -packed-fp32-ops tests/probes/e4m3_rate_probe.hip -o /tmp/e4m3_rate_probe
//   /tmp/e4m3_rate_probe
//
// Workgroups of 8 waves, one per compute unit (two waves per SIMD, as the large tiles of
// the linear).  A wave holds the operands of a 128 x 64 sub-tile with K 128 (8 x 4 tiles of
// 16 x 16, or 4 x 2 of 32 x 32 with two steps of 64) and multiplies all pairs, over and
// over.  "chained": the MFMAs add to the 128 sums themselves; "+ fma": they start from
// zero and one fma per result joins it, scaled, to the sum.  Codes are normal (a third of
// the largest code) or zero: the difference is the chip's power.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

#define CK(x)                                                                    \
  do {                                                                           \
    hipError_t e_ = (x);                                                         \
    if (e_ != hipSuccess) {                                                      \
      std::printf("HIP error %s at line %d\n", hipGetErrorString(e_), __LINE__); \
      return 1;                                                                  \
    }                                                                            \
  } while (0)

constexpr int kThreads = 512;  // 8 waves
constexpr int kFrags = 12;     // 8 of one operand, 4 of the other, 32 bytes per lane each

enum Mode { kSmall, kSmallFma, kBig };

// codes: kFrags fragments of kThreads lanes
template <Mode kMode>
__global__ __launch_bounds__(kThreads, 2) void mfma_kernel(const v8i* codes, int iters, float s, float* out) {
  v8i a[8], b[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = codes[i * kThreads + threadIdx.x];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = codes[(8 + j) * kThreads + threadIdx.x];
  float sum = 0.f;
  if constexpr (kMode != kBig) {
    v4f acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int it = 0; it < iters; ++it) {
      __asm__ volatile("" : "+v"(a[0]), "+v"(b[0]));
      if constexpr (kMode == kSmall) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], b[j], acc[i][j], 0, 0, 0, 0, 0, 0);
      } else {
        v4f t[2];
#pragma unroll
        for (int n = 0; n < 34; ++n) {  // results join two MFMAs later
          if (n >= 2) {
            const int m = n - 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m / 4][m % 4][e] = fmaf(t[m & 1][e], s, acc[m / 4][m % 4][e]);
          }
          if (n < 32)
            t[n & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[n / 4], b[n % 4], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                                        0, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += acc[i][j][0] + acc[i][j][1] + acc[i][j][2] + acc[i][j][3];
  } else {
    v16f acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    for (int it = 0; it < iters; ++it) {
      __asm__ volatile("" : "+v"(a[0]), "+v"(b[0]));
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[4 * k + i], b[2 * k + j], acc[i][j], 0, 0, 0, 0,
                                                                        0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum += acc[i][j][e];
  }
  out[blockIdx.x * kThreads + threadIdx.x] = sum;
}

// the nearest e4m3 code
uint8_t code_of(float v) {
  auto value = [](int c) { return c >> 3 ? std::ldexp(1.f + (c & 7) / 8.f, (c >> 3) - 7) : std::ldexp((c & 7) / 8.f, -6); };
  int best = 0;
  for (int c = 0; c < 127; ++c)
    if (std::fabs(value(c) - std::fabs(v)) < std::fabs(value(best) - std::fabs(v))) best = c;
  return (uint8_t)(best | (v < 0.f ? 128 : 0));
}

template <Mode kMode>
int run(const char* name, bool zero, const v8i* codes, int cus, float* out) {
  hipEvent_t e0, e1;
  CK(hipEventCreate(&e0));
  CK(hipEventCreate(&e1));
  const int iters = 20000;
  const double ops = 2.0 * 128 * 64 * 128 * 8 * (double)cus * iters;  // products and sums of a launch
  float best = 0.f, ms = 0.f;
  for (int rep = 0; rep < 4; ++rep) {
    CK(hipEventRecord(e0, 0));
    hipLaunchKernelGGL((mfma_kernel<kMode>), dim3(cus), dim3(kThreads), 0, 0, codes, iters, 1e-3f, out);
    CK(hipGetLastError());
    CK(hipEventRecord(e1, 0));
    CK(hipEventSynchronize(e1));
    CK(hipEventElapsedTime(&ms, e0, e1));
    if (rep > 0 && (best == 0.f || ms < best)) best = ms;
  }
  std::printf("mfma %s, %s codes: %7.3f ms  %5.2f PFLOP/s\n", name, zero ? "zero  " : "normal", best, ops / best / 1e12);
  std::fflush(stdout);
  return 0;
}

int main() {
  hipDeviceProp_t prop;
  CK(hipGetDeviceProperties(&prop, 0));
  const int cus = prop.multiProcessorCount;
  std::printf("compute units: %d\n", cus);
  v8i* codes;
  float* out;
  CK(hipMalloc(&codes, sizeof(v8i) * kFrags * kThreads));
  CK(hipMalloc(&out, sizeof(float) * cus * kThreads));
  std::mt19937 rng(1);
  std::normal_distribution<float> normal(0.f, 448.f / 3.f);
  for (int zero = 0; zero < 2; ++zero) {
    std::vector<uint8_t> h(sizeof(v8i) * kFrags * kThreads, 0);
    if (!zero)
      for (auto& v : h) v = code_of(normal(rng));
    CK(hipMemcpy(codes, h.data(), h.size(), hipMemcpyHostToDevice));
    if (run<kSmall>("f32 16x16x128 e4m3 chained", zero, codes, cus, out)) return 1;
    if (run<kSmallFma>("f32 16x16x128 e4m3 + fma  ", zero, codes, cus, out)) return 1;
    if (run<kBig>("f32 32x32x64  e4m3 chained", zero, codes, cus, out)) return 1;
  }
  CK(hipFree(codes));
  CK(hipFree(out));
  return 0;
}
