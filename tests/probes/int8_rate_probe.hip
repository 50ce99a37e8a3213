// What MI355X (gfx950) reaches on int8 matrix instructions fed from registers, and
// on a copy.  Not part of the library or the tests: a measurement program whose printed
// figures back the rates that the 8-bit linear and the row kernels are held against.
//
//   hipcc --offload-arch=gfx950 -O3 -std=c++17 -Xclang -target-feature \
//         -Xclang -packed-fp32-ops tests/probes/int8_rate_probe.hip -o /tmp/int8_rate_probe
//   /tmp/int8_rate_probe
//
//  * mfma: workgroups of 8 waves, one per compute unit (two waves per SIMD, as the
//    large tiles of the 8-bit linear).  A wave holds the operands of a 128 x 64 sub-tile
//    (8 x 4 tiles of 16 x 16, k 64, or 4 x 2 of 32 x 32, two k steps of 32: the same bytes
//    and products) and multiplies all pairs, over and over, into 128 int32 accumulators.
//    Codes are random (-127 .. 127) or zero: the difference is the chip's power.
//  * copy: 1 GiB, 16 bytes per lane, grid-stride.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <vector>

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

#define CK(x)                                                                    \
  do {                                                                           \
    hipError_t e_ = (x);                                                         \
    if (e_ != hipSuccess) {                                                      \
      std::printf("HIP error %s at line %d\n", hipGetErrorString(e_), __LINE__); \
      return 1;                                                                  \
    }                                                                            \
  } while (0)

constexpr int kThreads = 512;  // 8 waves
constexpr int kFrags = 12;     // 8 of one operand, 4 of the other, 16 bytes per lane each

// codes: kFrags fragments of kThreads lanes
template <bool kBig>
__global__ __launch_bounds__(kThreads, 2) void mfma_kernel(const v4i* codes, int iters, int* out) {
  v4i a[8], b[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = codes[i * kThreads + threadIdx.x];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = codes[(8 + j) * kThreads + threadIdx.x];
  int sum = 0;
  if constexpr (!kBig) {
    v4i acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    for (int it = 0; it < iters; ++it) {
      __asm__ volatile("" : "+v"(a[0]), "+v"(b[0]));
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += acc[i][j][0] ^ acc[i][j][3];
  } else {
    v16i acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
    for (int it = 0; it < iters; ++it) {
      __asm__ volatile("" : "+v"(a[0]), "+v"(b[0]));
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[4 * k + i], b[2 * k + j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) sum += acc[i][j][0] ^ acc[i][j][15];
  }
  out[blockIdx.x * kThreads + threadIdx.x] = sum;
}

__global__ __launch_bounds__(256) void copy_kernel(const uint4* src, uint4* dst, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) dst[i] = src[i];
}

int main() {
  hipDeviceProp_t prop;
  CK(hipGetDeviceProperties(&prop, 0));
  const int cus = prop.multiProcessorCount;
  std::printf("compute units: %d\n", cus);
  hipEvent_t e0, e1;
  CK(hipEventCreate(&e0));
  CK(hipEventCreate(&e1));
  v4i* codes;
  int* out;
  CK(hipMalloc(&codes, sizeof(v4i) * kFrags * kThreads));
  CK(hipMalloc(&out, sizeof(int) * cus * kThreads));
  const int iters = 20000;
  const double ops = 2.0 * 128 * 64 * 64 * 8 * (double)cus * iters;  // products and sums of a launch
  for (int zero = 0; zero < 2; ++zero) {
    std::vector<int8_t> h(sizeof(v4i) * kFrags * kThreads, 0);
    uint32_t s = 12345;
    if (!zero)
      for (auto& v : h) {
        s = s * 1664525u + 1013904223u;
        v = (int8_t)((int)((s >> 8) % 255u) - 127);
      }
    CK(hipMemcpy(codes, h.data(), h.size(), hipMemcpyHostToDevice));
    for (int big = 0; big < 2; ++big) {
      float best = 0.f, ms = 0.f;
      for (int rep = 0; rep < 4; ++rep) {
        CK(hipEventRecord(e0, 0));
        if (big) hipLaunchKernelGGL(mfma_kernel<true>, dim3(cus), dim3(kThreads), 0, 0, codes, iters, out);
        else hipLaunchKernelGGL(mfma_kernel<false>, dim3(cus), dim3(kThreads), 0, 0, codes, iters, out);
        CK(hipGetLastError());
        CK(hipEventRecord(e1, 0));
        CK(hipEventSynchronize(e1));
        CK(hipEventElapsedTime(&ms, e0, e1));
        if (rep > 0 && (best == 0.f || ms < best)) best = ms;
      }
      std::printf("mfma i32 %s i8, %s codes: %7.3f ms  %5.2f POP/s (last %5.2f)\n", big ? "32x32x32" : "16x16x64",
                  zero ? "zero  " : "random", best, ops / best / 1e12, ops / ms / 1e12);
    }
  }
  const size_t bytes = (size_t)1 << 30;
  uint4 *src, *dst;
  CK(hipMalloc(&src, bytes));
  CK(hipMalloc(&dst, bytes));
  hipLaunchKernelGGL(copy_kernel, dim3(cus * 16), dim3(256), 0, 0, dst, src, bytes / 16);
  for (int per_cu = 8; per_cu <= 64; per_cu *= 2) {
    CK(hipEventRecord(e0, 0));
    for (int k = 0; k < 20; ++k)
      hipLaunchKernelGGL(copy_kernel, dim3(cus * per_cu), dim3(256), 0, 0, src, dst, bytes / 16);
    CK(hipGetLastError());
    CK(hipEventRecord(e1, 0));
    CK(hipEventSynchronize(e1));
    float ms = 0.f;
    CK(hipEventElapsedTime(&ms, e0, e1));
    std::printf("copy 1 GiB, %2d workgroups per compute unit: %6.1f us  %5.2f TB/s (read and written)\n", per_cu,
                ms / 20 * 1e3, 2.0 * bytes / (ms / 20) / 1e9);
  }
  CK(hipFree(src));
  CK(hipFree(dst));
  CK(hipFree(codes));
  CK(hipFree(out));
  return 0;
}
