// Drives the C ABI of the block operators and the 8-bit packer under
// AddressSanitizer and UndefinedBehaviorSanitizer, against the fake runtime.
// Modes as in driver.cpp: full, arch-mismatch, no-device.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <string>
#include <vector>

#include "svdq.h"
#include "fake_runtime.h"

static int g_failures = 0;
#define CHECK(cond)                                                                                        \
  do {                                                                                                     \
    if (!(cond)) {                                                                                         \
      std::fprintf(stderr, "%s:%d: CHECK failed: %s (last error: %s)\n", __FILE__, __LINE__, #cond,        \
                   svdq_last_error());                                                                     \
      ++g_failures;                                                                                        \
    }                                                                                                      \
  } while (0)

static void* at(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 40); }

static void run_calls(svdq_status want) {
  const int64_t axes[3] = {16, 56, 56};
  float* f[12];
  for (int i = 0; i < 12; ++i) f[i] = static_cast<float*>(at(i));
  int8_t* c = static_cast<int8_t*>(at(20));
  CHECK(svdq_quantize_act_int8(at(1), f[2], 5, 128, c, f[4], nullptr) == want);
  CHECK(svdq_w8a8_gemm(c, f[2], static_cast<int8_t*>(at(3)), f[4], nullptr, 5, 128, 192, 0, at(6), nullptr, 0,
                       nullptr) == want);
  CHECK(svdq_gate_norm_modulate(at(1), 0, 128, at(2), 128, 2, at(3), at(4), 2, 384, 1.f, 1, at(5), at(6), at(7), 2, 384,
                                1e-6f, 4, 128, at(8), 128, 1, f[9], at(10), f[11], nullptr) == want);
  CHECK(svdq_rope_axes_tables(at(1), 0, 7, 3, axes, 1e4, 0, f[2], f[3], nullptr) == want);
  if (want == SVDQ_STATUS_SUCCESS) CHECK(g_fake.last_window[0] == 64);
  CHECK(svdq_rope_axes(at(1), 3072, 8, at(2), 3072, 2, 128, 6, at(3), 1, 3, 3, axes, 1e4, 1, 1, at(4), at(5), 1e-6f, at(6),
                       1024, at(7), 256, nullptr) == want);
}

static void full_mode() {
  g_fake.launches = 0;
  run_calls(SVDQ_STATUS_SUCCESS);
  CHECK(g_fake.launches == 5);
  CHECK(svdq_last_error()[0] == 0);
  // the extremes of the sizes: no overflow in the range checks
  const int64_t big[2] = {std::numeric_limits<int64_t>::max() - 1, std::numeric_limits<int64_t>::max() - 1};
  CHECK(svdq_rope_axes_tables(at(1), 0, 7, 2, big, 1e4, 0, static_cast<float*>(at(2)), static_cast<float*>(at(3)),
                              nullptr) == SVDQ_STATUS_NOT_SUPPORTED);
  const int64_t w = 1ll << 24;
  CHECK(svdq_quantize_act_int8(at(1), nullptr, w, 65536, static_cast<int8_t*>(at(100)), static_cast<float*>(at(50)),
                               nullptr) == SVDQ_STATUS_SUCCESS);
  const int64_t m = std::numeric_limits<int64_t>::max();
  CHECK(svdq_w8a8_gemm(nullptr, nullptr, nullptr, nullptr, nullptr, m, 64, 64, 0, nullptr, nullptr, 0, nullptr) ==
        SVDQ_STATUS_NOT_SUPPORTED);
  CHECK(svdq_w8a8_gemm_workspace_size(m, m, m) == 0);
  CHECK(svdq_gate_norm_modulate(at(1), 0, m, nullptr, 0, 0, nullptr, nullptr, 0, 0, 1.f, 1, nullptr, nullptr, nullptr, 0, 0,
                                0.f, 4, 128, nullptr, 0, 0, nullptr, at(9), nullptr, nullptr) != SVDQ_STATUS_SUCCESS);
  g_fake.gemm_need = 4096;
  CHECK(svdq_w8a8_gemm(static_cast<int8_t*>(at(1)), static_cast<float*>(at(2)), static_cast<int8_t*>(at(3)),
                       static_cast<float*>(at(4)), nullptr, 5, 64, 64, 0, at(6), at(7), 4096, nullptr) ==
        SVDQ_STATUS_SUCCESS);
  CHECK(g_fake.last_ws_bytes == 4096);
  g_fake.gemm_need = 0;

  // the packer on buffers of exactly its sizes
  const int64_t N = 37, K = 51;
  std::vector<uint16_t> wb(N * K);
  for (size_t i = 0; i < wb.size(); ++i) wb[i] = static_cast<uint16_t>(0x3C00 + (i * 2654435761u >> 20) % 900 + (i % 3 ? 0 : 0x8000));
  std::vector<float> lam(K, 0.5f);
  std::vector<int8_t> q(N * K);
  std::vector<float> s(N);
  CHECK(svdq_pack_weights_int8(wb.data(), lam.data(), N, K, q.data(), s.data()) == SVDQ_STATUS_SUCCESS);
  CHECK(svdq_pack_weights_int8(wb.data(), nullptr, N, K, q.data(), s.data()) == SVDQ_STATUS_SUCCESS);
  for (float v : s) CHECK(std::isfinite(v) && v > 0);
  wb[77] = 0x7FC0;
  CHECK(svdq_pack_weights_int8(wb.data(), nullptr, N, K, q.data(), s.data()) == SVDQ_STATUS_INVALID_VALUE);
  CHECK(svdq_pack_weights_int8(nullptr, nullptr, N, K, q.data(), s.data()) == SVDQ_STATUS_INVALID_VALUE);
  CHECK(svdq_pack_weights_int8(wb.data(), nullptr, 0, K, q.data(), s.data()) == SVDQ_STATUS_INVALID_VALUE);
}

int main(int argc, char** argv) {
  const std::string mode = argc > 1 ? argv[1] : "full";
  g_fake.gemm_need = 0;
  if (mode == "full") {
    full_mode();
  } else {
    g_fake.launches = 0;
    run_calls(mode == "arch-mismatch" ? SVDQ_STATUS_ARCH_MISMATCH : SVDQ_STATUS_NO_DEVICE);
    CHECK(g_fake.launches == 0);
  }
  if (g_failures) return 1;
  std::printf("host checks passed: %s\n", mode.c_str());
  return 0;
}
