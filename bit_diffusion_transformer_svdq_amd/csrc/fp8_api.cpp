// C ABI of the 8-bit floating-point linear (e4m3 codes, a scale for each block of 128)
// and of the gated feed-forward product on it (declarations and the contract:
// include/svdq.h).  Arguments are checked before any HIP call, as in api.cpp.

#include "api_checks.h"
#include "svdq_internal.h"

namespace {

using namespace svdq_api;

constexpr int64_t kMaxStride = 1ll << 37;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

svdq_status validate(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0)
    return fail(SVDQ_STATUS_INVALID_VALUE, "bad dims M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (K % 64 != 0) return fail(SVDQ_STATUS_NOT_SUPPORTED, "K=%lld is not a multiple of 64", (long long)K);
  if (N % 64 != 0) return fail(SVDQ_STATUS_NOT_SUPPORTED, "N=%lld is not a multiple of 64", (long long)N);
  if (M > kMaxRows || N > (1ll << 20) || K > svdq::kInt8MaxK)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "problem too large M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                (long long)K);
  return SVDQ_STATUS_SUCCESS;
}

// rows of M scales, one row per block of `width` channels; the stride of a single row is not read
svdq_status check_stride(int64_t stride, int64_t M, int64_t width, const char* name) {
  if (blocks(width) == 1) return SVDQ_STATUS_SUCCESS;
  if (stride < M)
    return fail(SVDQ_STATUS_INVALID_VALUE, "%s: stride %lld is smaller than M=%lld", name, (long long)stride, (long long)M);
  if (stride > kMaxStride) return fail(SVDQ_STATUS_NOT_SUPPORTED, "%s: a stride above 2^37", name);
  return SVDQ_STATUS_SUCCESS;
}

Rows scale_rows(const float* p, int64_t stride, int64_t M, int64_t width, const char* name) {
  const bool one = blocks(width) == 1;
  return Rows{p, one ? 0 : sz(stride, 4), sz(M, 4), (size_t)blocks(width), name};
}

// the scales of a run of tokens may start at any of them
bool bad_scales(const float* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

Rows flat(const void* p, size_t bytes, const char* name) { return Rows{p, 0, bytes, 1, name}; }

svdq::Fp8Args sizes(int64_t M, int64_t N, int64_t K, bool gated, bool coded) {
  // (the plan asks of the pointers only whether they are null)
  static const uint8_t some_codes = 0;
  static float some_scale = 0.f;
  svdq::Fp8Args a{};
  a.M = (int)M, a.N = (int)N, a.K = (int)K;
  a.up = gated ? &some_codes : nullptr;
  a.out_scales = coded ? &some_scale : nullptr;
  return a;
}

svdq_status run(const svdq::Fp8Args& a, void* workspace, size_t workspace_bytes, size_t need, const char* query,
                void* stream, const char* what) {
  const bool gated = a.up != nullptr, coded = a.out_scales != nullptr;
  for (const void* p : {(const void*)a.act, (const void*)a.w, (const void*)a.w_scales, (const void*)a.up,
                        (const void*)a.up_scales, (const void*)a.bias, (const void*)a.up_bias, (const void*)a.smooth,
                        (const void*)a.out})
    if (bad_ptr(p)) return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  if (bad_scales(a.act_scales) || bad_scales(a.out_scales))
    return fail(SVDQ_STATUS_INVALID_VALUE, "token scales must be 4-byte aligned");
  svdq_status s = check_workspace(workspace, workspace_bytes, need, query);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  const size_t wb = sz(a.N, a.K), sb = sz(blocks(a.N), blocks(a.K), 4);
  const Rows out = flat(a.out, sz(a.M, a.N, coded ? 1 : 2), gated ? "out" : "y"),
             scales = coded ? scale_rows(a.out_scales, a.out_stride, a.M, a.N, "out_scales") : Rows{},
             ws = flat(need ? workspace : nullptr, need, "workspace"),
             act = flat(a.act, sz(a.M, a.K), "act_codes"),
             as = scale_rows(a.act_scales, a.act_stride, a.M, a.K, "act_scales"),
             w = flat(a.w, wb, gated ? "gate_codes" : "w_codes"),
             wsc = flat(a.w_scales, sb, gated ? "gate_scales" : "w_scales"),
             up = flat(a.up, wb, "up_codes"), usc = flat(a.up_scales, sb, "up_scales"),
             b = flat(a.bias, sz(a.N, 2), gated ? "gate_bias" : "bias"), ub = flat(a.up_bias, sz(a.N, 2), "up_bias"),
             sm = flat(a.smooth, sz(a.N, 4), "smooth");
  s = check_rows(out, {act, as, w, wsc, up, usc, b, ub, sm, scales, ws});
  if (s == SVDQ_STATUS_SUCCESS) s = check_rows(scales, {act, as, w, wsc, up, usc, b, ub, sm, ws});
  if (s == SVDQ_STATUS_SUCCESS) s = check_rows(ws, {act, as, w, wsc, up, usc, b, ub, sm});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  return launched(svdq::launch_fp8_gemm(a, svdq::Workspace{workspace, workspace_bytes},
                                        static_cast<hipStream_t>(stream)), what);
}

}  // namespace

extern "C" {

svdq_status svdq_quantize_act_fp8(const void* x, const float* smooth, int64_t M, int64_t K, void* act_codes,
                                  float* act_scales, int64_t act_scale_stride, void* stream) {
  svdq_status s = validate(M, 64, K);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (M == 0) return ok();
  if (!x || !act_codes || !act_scales) return fail(SVDQ_STATUS_INVALID_VALUE, "null x/act_codes/act_scales");
  s = check_stride(act_scale_stride, M, K, "act_scales");
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (bad_ptr(x) || bad_ptr(smooth) || bad_ptr(act_codes))
    return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  if (bad_scales(act_scales)) return fail(SVDQ_STATUS_INVALID_VALUE, "token scales must be 4-byte aligned");
  const Rows codes = flat(act_codes, sz(M, K), "act_codes"),
             scales = scale_rows(act_scales, act_scale_stride, M, K, "act_scales"), rx = flat(x, sz(M, K, 2), "x"),
             sm = flat(smooth, sz(K, 4), "smooth");
  s = check_rows(codes, {rx, sm, scales});
  if (s == SVDQ_STATUS_SUCCESS) s = check_rows(scales, {rx, sm});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  const svdq::QuantFp8Args a{static_cast<const uint16_t*>(x), smooth, static_cast<uint8_t*>(act_codes), act_scales,
                             blocks(K) == 1 ? M : act_scale_stride, (int)M, (int)K};
  return launched(svdq::launch_quant_fp8(a, static_cast<hipStream_t>(stream)), "quantize fp8");
}

size_t svdq_fp8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (validate(M, N, K) != SVDQ_STATUS_SUCCESS || M == 0) return 0;
  return svdq::fp8_workspace_bytes(sizes(M, N, K, false, false));
}

size_t svdq_fp8_gated_gemm_workspace_size(int64_t M, int64_t F, int64_t K, int out_type) {
  if (validate(M, F, K) != SVDQ_STATUS_SUCCESS || M == 0) return 0;
  if (out_type != SVDQ_GATED_OUT_BF16 && out_type != SVDQ_GATED_OUT_FP8) return 0;
  return svdq::fp8_workspace_bytes(sizes(M, F, K, true, out_type == SVDQ_GATED_OUT_FP8));
}

svdq_status svdq_debug_set_fp8_plan(int tile, int splits) {
  if (!svdq::fp8_tile_known(tile)) return fail(SVDQ_STATUS_INVALID_VALUE, "unknown fp8 tile %d", tile);
  if (splits < 0 || splits > 16) return fail(SVDQ_STATUS_INVALID_VALUE, "bad split count %d (0..16)", splits);
  svdq::set_fp8_plan_override(tile, splits);
  return ok();
}

svdq_status svdq_fp8_gemm(const void* act_codes, const float* act_scales, int64_t act_scale_stride,
                          const void* w_codes, const float* w_scales, const void* bias, int64_t M, int64_t N, int64_t K,
                          int epilogue, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  svdq_status s = validate(M, N, K);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (epilogue != SVDQ_EPILOGUE_NONE && epilogue != SVDQ_EPILOGUE_GELU_TANH)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown epilogue %d", epilogue);
  if (M == 0) return ok();
  if (!act_codes || !act_scales || !w_codes || !w_scales || !y)
    return fail(SVDQ_STATUS_INVALID_VALUE, "null act_codes/act_scales/w_codes/w_scales/y");
  s = check_stride(act_scale_stride, M, K, "act_scales");
  if (s != SVDQ_STATUS_SUCCESS) return s;
  svdq::Fp8Args a = sizes(M, N, K, false, false);
  const size_t need = svdq::fp8_workspace_bytes(a);
  a.act = static_cast<const uint8_t*>(act_codes);
  a.act_scales = act_scales;
  a.act_stride = blocks(K) == 1 ? M : act_scale_stride;
  a.w = static_cast<const uint8_t*>(w_codes);
  a.w_scales = w_scales;
  a.bias = static_cast<const uint16_t*>(bias);
  a.out = y;
  a.epilogue = epilogue == SVDQ_EPILOGUE_GELU_TANH ? svdq::kEpilogueGelu : svdq::kEpilogueNone;
  return run(a, workspace, workspace_bytes, need, "svdq_fp8_gemm_workspace_size", stream, "fp8 gemm");
}

svdq_status svdq_fp8_gated_gemm(const void* act_codes, const float* act_scales, int64_t act_scale_stride,
                                const void* gate_codes, const float* gate_scales, const void* up_codes,
                                const float* up_scales, const void* gate_bias, const void* up_bias, int64_t M, int64_t F,
                                int64_t K, int activation, int out_type, const float* smooth, void* out,
                                float* out_scales, int64_t out_scale_stride, void* workspace, size_t workspace_bytes,
                                void* stream) {
  svdq_status s = validate(M, F, K);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (activation != SVDQ_ACT_SILU && activation != SVDQ_ACT_GELU_TANH)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown activation %d", activation);
  if (out_type != SVDQ_GATED_OUT_BF16 && out_type != SVDQ_GATED_OUT_FP8)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown output type %d", out_type);
  const bool coded = out_type == SVDQ_GATED_OUT_FP8;
  if (smooth && !coded) return fail(SVDQ_STATUS_INVALID_VALUE, "smooth needs the 8-bit output");
  if (M == 0) return ok();
  if (!act_codes || !act_scales || !gate_codes || !gate_scales || !up_codes || !up_scales || !out || (coded && !out_scales))
    return fail(SVDQ_STATUS_INVALID_VALUE,
                "null act_codes/act_scales/gate_codes/gate_scales/up_codes/up_scales/out/out_scales");
  s = check_stride(act_scale_stride, M, K, "act_scales");
  if (s == SVDQ_STATUS_SUCCESS && coded) s = check_stride(out_scale_stride, M, F, "out_scales");
  if (s != SVDQ_STATUS_SUCCESS) return s;
  svdq::Fp8Args a = sizes(M, F, K, true, coded);
  const size_t need = svdq::fp8_workspace_bytes(a);
  a.act = static_cast<const uint8_t*>(act_codes);
  a.act_scales = act_scales;
  a.act_stride = blocks(K) == 1 ? M : act_scale_stride;
  a.w = static_cast<const uint8_t*>(gate_codes);
  a.w_scales = gate_scales;
  a.up = static_cast<const uint8_t*>(up_codes);
  a.up_scales = up_scales;
  a.bias = static_cast<const uint16_t*>(gate_bias);
  a.up_bias = static_cast<const uint16_t*>(up_bias);
  a.smooth = smooth;
  a.out = out;
  a.out_scales = coded ? out_scales : nullptr;
  a.out_stride = blocks(F) == 1 ? M : out_scale_stride;
  a.epilogue = activation == SVDQ_ACT_SILU ? svdq::kActSilu : svdq::kActGelu;
  return run(a, workspace, workspace_bytes, need, "svdq_fp8_gated_gemm_workspace_size", stream, "fp8 gated gemm");
}

}  // extern "C"
