// Stand-ins for the launchers of the block operators (see fake_runtime.cpp):
// each records its call; the 8-bit linear's workspace need is set by the driver.
#include "svdq_internal.h"
#include "fake_runtime.h"

namespace svdq {

static hipError_t record(const char* name, const void* out) {
  ++g_fake.launches;
  g_fake.last = name;
  g_fake.last_out = out;
  return hipSuccess;
}

hipError_t launch_gate_norm(const GateNormArgs& a, hipStream_t) { return record("gate_norm", a.z ? a.z : a.h); }
hipError_t launch_quant_int8(const QuantInt8Args& a, hipStream_t) { return record("quant_int8", a.codes); }
size_t w8a8_workspace_bytes(int64_t, int64_t, int64_t) { return g_fake.gemm_need; }
hipError_t launch_w8a8_gemm(const W8a8Args& a, Workspace ws, hipStream_t) {
  g_fake.last_ws_bytes = ws.bytes;
  return record("w8a8", a.y);
}
bool w8a8_tile_known(int tile) { return tile == 0; }
void set_w8a8_plan_override(int, int) {}
hipError_t launch_rope_tables(const void*, bool, const RopeAxes& x, int64_t, float* cos, float*, hipStream_t) {
  g_fake.last_window[0] = x.half;
  return record("tables", cos);
}
hipError_t launch_rope_axes(const RopeArgs& a, const RopeAxes&, bool, hipStream_t) { return record("rope", a.q_out); }

}  // namespace svdq
