// How the matrix core of MI355X (gfx950) adds e4m3 products.  Not part of the library or the
// tests: a measurement program whose printed figures back what the 8-bit floating-point
// linear's kernels, header and tests say of their sums.
//
//   hipcc --offload-arch=gfx950 -O2 -std=c++17 -Xclang -target-feature
//         -Xclang -packed-fp32-ops tests/probes/e4m3_sum_probe.hip -o /tmp/e4m3_sum_probe
//   /tmp/e4m3_sum_probe
//
// One wave runs one MFMA whose row 0 and column 0 hold a few powers of two, all else
// zero; its element (0, 0) tells which of them the sum keeps:
//  * big, -big and a small product at three places of K: the smallest product that is
//    kept beside the big one, in its group of eight neighbours and outside of it;
//  * a small product of either sign beside a big one of either sign: which way it is cut;
//  * products of subnormal codes and of the largest ones: which exponent decides.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kRows = 16, kK = 128;

__global__ void mfma16(const uint8_t* a, const uint8_t* b, float* d) {
  const int r = threadIdx.x & 15, q = threadIdx.x >> 4;
  v8i x, y;
  for (int e = 0; e < 8; ++e) {
    x[e] = reinterpret_cast<const int*>(a + r * kK + 32 * q)[e];
    y[e] = reinterpret_cast<const int*>(b + r * kK + 32 * q)[e];
  }
  const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
  if (threadIdx.x == 0) d[0] = p[0];
}

__global__ void mfma32(const uint8_t* a, const uint8_t* b, float* d) {
  const int r = threadIdx.x & 31, q = threadIdx.x >> 5;
  v8i x, y;
  for (int e = 0; e < 8; ++e) {
    x[e] = r < kRows ? reinterpret_cast<const int*>(a + r * kK + 32 * q)[e] : 0;
    y[e] = r < kRows ? reinterpret_cast<const int*>(b + r * kK + 32 * q)[e] : 0;
  }
  v16f z;
  for (int e = 0; e < 16; ++e) z[e] = 0.f;
  const v16f p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, z, 0, 0, 0, 0, 0, 0);
  if (threadIdx.x == 0) d[0] = p[0];
}

__global__ void mfma16k32(const uint8_t* a, const uint8_t* b, float* d) {
  const int r = threadIdx.x & 15, q = threadIdx.x >> 4;
  const long x = *reinterpret_cast<const long*>(a + r * kK + 8 * q), y = *reinterpret_cast<const long*>(b + r * kK + 8 * q);
  const v4f p = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(x, y, v4f{0, 0, 0, 0}, 0, 0, 0);
  if (threadIdx.x == 0) d[0] = p[0];
}

// the code of +-2^e, e in -9 .. 8
static uint8_t pow2(int e, bool neg = false) {
  return static_cast<uint8_t>((e >= -6 ? (e + 7) << 3 : 1 << (e + 9)) | (neg ? 128 : 0));
}

struct Sum {
  std::vector<uint8_t> a = std::vector<uint8_t>(kRows * kK), b = a;
  uint8_t *da = nullptr, *db = nullptr;
  float* dd = nullptr;
  Sum() {
    if (hipMalloc(&da, a.size()) != hipSuccess || hipMalloc(&db, b.size()) != hipSuccess || hipMalloc(&dd, 4) != hipSuccess) std::exit(1);
  }
  void clear() { std::fill(a.begin(), a.end(), 0), std::fill(b.begin(), b.end(), 0); }
  void put(int k, int e, bool neg = false) {  // the product +-2^e at place k
    const int h = std::max(-9, std::min(8, e / 2));
    a[k] = pow2(h, neg), b[k] = pow2(e - h);
  }
  template <class K>
  float run(K kernel) {
    float v = 0.f;
    if (hipMemcpy(da, a.data(), a.size(), hipMemcpyHostToDevice) != hipSuccess) std::exit(1);
    if (hipMemcpy(db, b.data(), b.size(), hipMemcpyHostToDevice) != hipSuccess) std::exit(1);
    hipLaunchKernelGGL(kernel, dim3(1), dim3(64), 0, 0, da, db, dd);
    if (hipMemcpy(&v, dd, 4, hipMemcpyDeviceToHost) != hipSuccess) std::exit(1);
    return v;
  }
};

template <class K>
static void kept(Sum& s, const char* name, K kernel) {
  const int places[][3] = {{0, 1, 2}, {0, 1, 7}, {0, 16, 1}, {0, 1, 8}, {0, 16, 8}, {0, 1, 31}};
  for (const auto& p : places) {
    std::printf("%-12s big at %2d, -big at %2d, small at %2d: kept down to", name, p[0], p[1], p[2]);
    for (int big : {16, 8, 0}) {
      int last = big;
      for (int e = big; e >= -18; --e) {
        s.clear();
        s.put(p[0], big), s.put(p[1], big, true), s.put(p[2], e);
        if (s.run(kernel) != std::ldexp(1.f, e)) break;
        last = e;
      }
      std::printf("  2^%d (big 2^%d)", last, big);
    }
    std::printf("\n");
    std::fflush(stdout);
  }
}

int main() {
  Sum s;
  kept(s, "16x16x128", mfma16);
  kept(s, "32x32x64", mfma32);
  kept(s, "16x16x32", mfma16k32);
  for (int e = 4; e >= 1; --e)
    for (int sign = 0; sign < 4; ++sign) {
      s.clear();
      s.put(0, 16, sign & 1), s.put(1, e, sign & 2);
      std::printf("%s2^16 %s 2^%d = %.9g\n", sign & 1 ? "-" : "", sign & 2 ? "-" : "+", e, s.run(mfma16));
    }
  for (int e = 5; e >= 2; --e) {  // 8 significant bits: 1.265625 = 1.125^2
    s.clear();
    s.put(0, 16), s.put(1, e);
    s.a[1] |= 1, s.b[1] |= 1;
    std::printf("2^16 + 1.265625 2^%d = 2^16 + %.9g\n", e, s.run(mfma16) - 65536.f);
  }
  for (int e = -10; e >= -13; --e) {  // the codes' exponents 8 and -6, whose sum is 2, decide, not the product's own -1
    s.clear();
    s.a[0] = pow2(8), s.b[0] = pow2(-9);
    s.put(1, e);
    std::printf("2^8 2^-9 + 2^%d = 2^-1 + %.9g\n", e, s.run(mfma16) - 0.5f);
  }
  for (int e = 4; e >= 2; --e) {
    s.clear();
    s.a[0] = s.b[0] = 0x7E;
    s.put(1, e);
    std::printf("448^2 + 2^%d = 448^2 + %.9g\n", e, s.run(mfma16) - 200704.f);
  }
  return 0;
}
