// Drives the C ABI of the 8-bit floating-point linear, of the gated product and their
// packer under AddressSanitizer and UndefinedBehaviorSanitizer, against the fake runtime.
// Modes as in driver.cpp: full, arch-mismatch, no-device.
#include <cmath>
#include <cstdint>
#include <cstdio>
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
static float* f(int i) { return static_cast<float*>(at(i)); }

static void run_calls(svdq_status want) {
  const bool good = want == SVDQ_STATUS_SUCCESS;
  CHECK(svdq_quantize_act_fp8(at(1), f(2), 5, 192, at(3), f(4), 9, nullptr) == want);
  if (good) CHECK(g_fake.last_window[0] == 9);
  CHECK(svdq_quantize_act_fp8(at(1), nullptr, 5, 128, at(3), f(4), -1, nullptr) == want);
  if (good) CHECK(g_fake.last_window[0] == 5);  // the stride of one row is not read
  CHECK(svdq_fp8_gemm(at(1), f(2), 8, at(3), f(4), nullptr, 5, 128, 192, 0, at(6), nullptr, 0, nullptr) == want);
  if (good) CHECK(g_fake.last_window[0] == 0 && g_fake.last_window[1] == 0);
  for (int out : {0, 1}) {
    CHECK(svdq_fp8_gated_gemm(at(1), f(2), 5, at(3), f(4), at(5), f(6), at(7), nullptr, 5, 128, 192, 1, out, out ? f(8) : nullptr,
                              at(9), f(10), 5, nullptr, 0, nullptr) == want);
    if (good) CHECK(g_fake.last_window[0] == 1 && g_fake.last_window[1] == out);
  }
}

static void full_mode() {
  g_fake.launches = 0;
  run_calls(SVDQ_STATUS_SUCCESS);
  CHECK(g_fake.launches == 5);
  CHECK(svdq_last_error()[0] == 0);
  // the extremes of the sizes: no overflow in the range checks
  const int64_t m = std::numeric_limits<int64_t>::max(), w = 1ll << 24, far = 1ll << 37;
  CHECK(svdq_quantize_act_fp8(at(1), nullptr, w, 65536, at(100), f(300), far, nullptr) == SVDQ_STATUS_SUCCESS);
  CHECK(svdq_quantize_act_fp8(at(1), nullptr, w, 65536, at(100), f(300), m, nullptr) == SVDQ_STATUS_NOT_SUPPORTED);
  CHECK(svdq_fp8_gemm(nullptr, nullptr, 0, nullptr, nullptr, nullptr, m, 64, 64, 0, nullptr, nullptr, 0, nullptr) ==
        SVDQ_STATUS_NOT_SUPPORTED);
  CHECK(svdq_fp8_gemm_workspace_size(m, m, m) == 0 && svdq_fp8_gated_gemm_workspace_size(m, 64, 64, 0) == 0);
  CHECK(svdq_fp8_gated_gemm(at(1), f(2), m, at(3), f(4), at(5), f(6), nullptr, nullptr, 5, 128, 192, 0, 0, nullptr, at(9),
                            nullptr, 0, nullptr, 0, nullptr) == SVDQ_STATUS_NOT_SUPPORTED);
  CHECK(svdq_fp8_gemm(at(1), f(2), far, at(100), f(300), nullptr, w, 1 << 20, 65536, 0, at(700), nullptr, 0, nullptr) ==
        SVDQ_STATUS_SUCCESS);
  g_fake.gemm_need = 4096;
  CHECK(svdq_fp8_gemm(at(1), f(2), 5, at(3), f(4), nullptr, 5, 64, 192, 0, at(6), at(7), 4096, nullptr) == SVDQ_STATUS_SUCCESS);
  CHECK(g_fake.last_ws_bytes == 4096);
  CHECK(svdq_fp8_gemm(at(1), f(2), 5, at(3), f(4), nullptr, 5, 64, 192, 0, at(6), at(7), 4095, nullptr) == SVDQ_STATUS_INVALID_VALUE);
  g_fake.gemm_need = 0;

  // the packer on buffers of exactly its sizes
  for (int64_t N : {1, 128, 129, 300})
    for (int64_t K : {1, 51, 128, 257}) {
      std::vector<uint16_t> wb(N * K);
      for (size_t i = 0; i < wb.size(); ++i)
        wb[i] = static_cast<uint16_t>(0x3C00 + (i * 2654435761u >> 20) % 900 + (i % 3 ? 0 : 0x8000));
      std::vector<float> lam(K, 0.5f), s(((N + 127) / 128) * ((K + 127) / 128));
      std::vector<uint8_t> q(N * K);
      CHECK(svdq_pack_weights_fp8(wb.data(), lam.data(), N, K, q.data(), s.data()) == SVDQ_STATUS_SUCCESS);
      CHECK(svdq_pack_weights_fp8(wb.data(), nullptr, N, K, q.data(), s.data()) == SVDQ_STATUS_SUCCESS);
      for (float v : s) CHECK(std::isfinite(v) && v > 0);
      for (uint8_t c : q) CHECK((c & 127) != 127);
      wb[wb.size() - 1] = 0x7FC0;
      CHECK(svdq_pack_weights_fp8(wb.data(), nullptr, N, K, q.data(), s.data()) == SVDQ_STATUS_INVALID_VALUE);
      CHECK(svdq_pack_weights_fp8(nullptr, nullptr, N, K, q.data(), s.data()) == SVDQ_STATUS_INVALID_VALUE);
      CHECK(svdq_pack_weights_fp8(wb.data(), nullptr, 0, K, q.data(), s.data()) == SVDQ_STATUS_INVALID_VALUE);
    }
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
