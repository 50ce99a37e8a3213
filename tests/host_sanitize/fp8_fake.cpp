// Stand-ins for the launchers of the 8-bit floating-point linear (see fake_runtime.cpp):
// each records its call; the products' workspace need is set by the driver.
#include "svdq_internal.h"
#include "fake_runtime.h"

namespace svdq {

static hipError_t record(const char* name, const void* out) {
  ++g_fake.launches;
  g_fake.last = name;
  g_fake.last_out = out;
  return hipSuccess;
}

hipError_t launch_quant_fp8(const QuantFp8Args& a, hipStream_t) {
  g_fake.last_window[0] = (int)a.scale_stride;
  return record("quant_fp8", a.codes);
}
size_t fp8_workspace_bytes(const Fp8Args&) { return g_fake.gemm_need; }
hipError_t launch_fp8_gemm(const Fp8Args& a, Workspace ws, hipStream_t) {
  g_fake.last_ws_bytes = ws.bytes;
  g_fake.last_window[0] = a.up != nullptr;
  g_fake.last_window[1] = a.out_scales != nullptr;
  return record("fp8", a.out);
}
bool fp8_tile_known(int tile) { return tile == 0; }
void set_fp8_plan_override(int, int) {}

}  // namespace svdq
