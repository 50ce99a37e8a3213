// C ABI of the operators around the 4-bit linears of a transformer block: the
// 8-bit linear, the gated residual norms and the rotary positions with several
// axes (declarations and the contract: include/svdq.h).  Arguments are checked
// before any HIP call, as in api.cpp.

#include <cmath>
#include <cstring>

#include "api_checks.h"
#include "svdq_internal.h"

namespace {

using namespace svdq_api;

constexpr int64_t kMaxRows = 1ll << 24;

// rows of `width` bytes, `stride` bytes apart
struct Rows {
  const void* p;
  size_t stride, width, rows;
  const char* name;
};

size_t extent(const Rows& r) { return r.rows == 0 ? 0 : (r.rows - 1) * r.stride + r.width; }

// Whether two sets of rows may share a byte.  Rows of one stride can interleave
// (the Q and K columns of one projection's output): their places within a
// stride decide.
bool meet(const Rows& a, const Rows& b) {
  if (!a.p || !b.p) return false;
  if (!overlap({a.p, extent(a), a.name}, {b.p, extent(b), b.name})) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const size_t d = (size_t)((b0 >= a0 ? (b0 - a0) % a.stride : a.stride - (a0 - b0) % a.stride) % a.stride);
  return d < a.width || d + b.width > a.stride;
}

svdq_status check_rows(const Rows& out, std::initializer_list<Rows> others) {
  for (const Rows& o : others)
    if (meet(out, o)) return fail(SVDQ_STATUS_INVALID_VALUE, "output %s overlaps %s", out.name, o.name);
  return SVDQ_STATUS_SUCCESS;
}

// `in` as check_rows takes it, or nothing where its rows are exactly those of
// `out`: an update in place, of an input that each thread reads at its own places
// before it writes them
Rows unless_in_place(const Rows& out, const Rows& in) {
  const bool same = in.p == out.p && in.width == out.width && in.rows == out.rows &&
                    (in.stride == out.stride || in.rows == 1);
  return same ? Rows{} : in;
}

bool bad_ptr(const void* p) { return p && !aligned16(p); }

svdq_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SVDQ_STATUS_HIP_ERROR, "%s launch: %s", what, hipGetErrorString(e));
  return ok();
}

svdq_status validate_w8a8(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0)
    return fail(SVDQ_STATUS_INVALID_VALUE, "bad dims M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (K % 64 != 0) return fail(SVDQ_STATUS_NOT_SUPPORTED, "K=%lld is not a multiple of 64", (long long)K);
  if (N % 64 != 0) return fail(SVDQ_STATUS_NOT_SUPPORTED, "N=%lld is not a multiple of 64", (long long)N);
  if (M > kMaxRows || N > (1ll << 20) || K > svdq::kInt8MaxK)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "problem too large M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                (long long)K);
  return SVDQ_STATUS_SUCCESS;
}

// axes, theta and spectrum -> RopeAxes
svdq_status read_axes(int64_t n_axes, const int64_t* axes, double theta, int spectrum, svdq::RopeAxes& x) {
  if (n_axes <= 0 || !axes) return fail(SVDQ_STATUS_INVALID_VALUE, "no axes");
  if (n_axes > svdq::kRopeMaxAxes)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "%lld axes (at most %d)", (long long)n_axes, svdq::kRopeMaxAxes);
  int64_t R = 0;
  x.n = (int)n_axes;
  for (int i = 0; i < x.n; ++i) {
    if (axes[i] <= 0 || axes[i] % 2 != 0)
      return fail(SVDQ_STATUS_INVALID_VALUE, "axis %d has width %lld (positive and even)", i, (long long)axes[i]);
    if (axes[i] > 2 * svdq::kRopeMaxAngles || (R += axes[i]) > 2 * svdq::kRopeMaxAngles)
      return fail(SVDQ_STATUS_NOT_SUPPORTED, "the axes are wider than %d channels", 2 * svdq::kRopeMaxAngles);
    x.width[i] = (int)axes[i];
  }
  if (!std::isfinite(theta) || theta <= 1.0) return fail(SVDQ_STATUS_INVALID_VALUE, "theta must be finite and > 1");
  if (spectrum != SVDQ_SPECTRUM_AXIS && spectrum != SVDQ_SPECTRUM_SHARED)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown spectrum %d", spectrum);
  x.half = (int)(R / 2);
  x.shared = spectrum == SVDQ_SPECTRUM_SHARED;
  x.theta = theta;
  return SVDQ_STATUS_SUCCESS;
}

bool known_positions(int t) { return t == SVDQ_POSITIONS_FP32 || t == SVDQ_POSITIONS_INT32; }

}  // namespace

extern "C" {

svdq_status svdq_quantize_act_int8(const void* x, const float* smooth, int64_t M, int64_t K, int8_t* act_codes,
                                   float* act_scales, void* stream) {
  svdq_status s = validate_w8a8(M, 64, K);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (M == 0) return ok();
  if (!x || !act_codes || !act_scales) return fail(SVDQ_STATUS_INVALID_VALUE, "null x/act_codes/act_scales");
  if (bad_ptr(x) || bad_ptr(smooth) || bad_ptr(act_codes) || bad_ptr(act_scales))
    return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  s = check_disjoint({{act_codes, sz(M, K), "act_codes"}, {act_scales, sz(M, 4), "act_scales"}},
                     {{x, sz(M, K, 2), "x"}, {smooth, sz(K, 4), "smooth"}});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  const svdq::QuantInt8Args a{static_cast<const uint16_t*>(x), smooth, act_codes, act_scales, (int)M, (int)K, 0};
  return launched(svdq::launch_quant_int8(a, static_cast<hipStream_t>(stream)), "quantize int8");
}

size_t svdq_w8a8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (validate_w8a8(M, N, K) != SVDQ_STATUS_SUCCESS || M == 0) return 0;
  return svdq::w8a8_workspace_bytes(M, N, K);
}

svdq_status svdq_debug_set_w8a8_plan(int tile, int splits) {
  if (!svdq::w8a8_tile_known(tile)) return fail(SVDQ_STATUS_INVALID_VALUE, "unknown w8a8 tile %d", tile);
  if (splits < 0 || splits > 16) return fail(SVDQ_STATUS_INVALID_VALUE, "bad split count %d (0..16)", splits);
  svdq::set_w8a8_plan_override(tile, splits);
  return ok();
}

svdq_status svdq_w8a8_gemm(const int8_t* act_codes, const float* act_scales, const int8_t* w_codes,
                           const float* w_scales, const void* bias, int64_t M, int64_t N, int64_t K, int epilogue,
                           void* y, void* workspace, size_t workspace_bytes, void* stream) {
  svdq_status s = validate_w8a8(M, N, K);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (epilogue != SVDQ_EPILOGUE_NONE && epilogue != SVDQ_EPILOGUE_GELU_TANH)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown epilogue %d", epilogue);
  if (M == 0) return ok();
  if (!act_codes || !act_scales || !w_codes || !w_scales || !y)
    return fail(SVDQ_STATUS_INVALID_VALUE, "null act_codes/act_scales/w_codes/w_scales/y");
  if (bad_ptr(act_codes) || bad_ptr(act_scales) || bad_ptr(w_codes) || bad_ptr(w_scales) || bad_ptr(bias) || bad_ptr(y))
    return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  const size_t need = svdq::w8a8_workspace_bytes(M, N, K);
  s = check_workspace(workspace, workspace_bytes, need, "svdq_w8a8_gemm_workspace_size");
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_disjoint({{y, sz(M, N, 2), "y"}, {need ? workspace : nullptr, need, "workspace"}},
                     {{act_codes, sz(M, K), "act_codes"}, {act_scales, sz(M, 4), "act_scales"},
                      {w_codes, sz(N, K), "w_codes"}, {w_scales, sz(N, 4), "w_scales"}, {bias, sz(N, 2), "bias"}});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  const svdq::W8a8Args a{act_codes, act_scales, w_codes, w_scales, static_cast<const uint16_t*>(bias),
                         static_cast<uint16_t*>(y), (int)M, (int)N, (int)K, epilogue};
  return launched(svdq::launch_w8a8_gemm(a, svdq::Workspace{workspace, workspace_bytes},
                                         static_cast<hipStream_t>(stream)), "w8a8 gemm");
}

svdq_status svdq_gate_norm_modulate(const void* x, int stream_type, int64_t x_stride, const void* y, int64_t y_stride,
                                    int post_norm, const void* post_weight, const void* gate, int64_t gate_rows,
                                    int64_t gate_stride, float residual_scale, int norm, const void* weight,
                                    const void* scale, const void* shift, int64_t mod_rows, int64_t mod_stride,
                                    float eps, int64_t M, int64_t C, void* h, int64_t h_stride, int out_type,
                                    const float* smooth, void* z, float* z_scales, void* stream) {
  if (M < 0 || C <= 0)
    return fail(SVDQ_STATUS_INVALID_VALUE, "bad dims M=%lld C=%lld", (long long)M, (long long)C);
  if (C % 8 != 0) return fail(SVDQ_STATUS_NOT_SUPPORTED, "C=%lld is not a multiple of 8", (long long)C);
  if (M > kMaxRows || C > svdq::kGateNormMaxC)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "problem too large M=%lld C=%lld", (long long)M, (long long)C);
  if (stream_type != SVDQ_STREAM_BF16 && stream_type != SVDQ_STREAM_FP32)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown stream type %d", stream_type);
  for (int n : {post_norm, norm})
    if (n != SVDQ_NORM_NONE && n != SVDQ_NORM_LAYER && n != SVDQ_NORM_RMS)
      return fail(SVDQ_STATUS_INVALID_VALUE, "unknown norm %d", n);
  if (out_type != SVDQ_NORM_OUT_BF16 && out_type != SVDQ_NORM_OUT_INT8)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown output type %d", out_type);
  const bool q8 = out_type == SVDQ_NORM_OUT_INT8;
  if (q8 && C % 64 != 0)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "C=%lld is not a multiple of 64 (8-bit output)", (long long)C);
  if (!std::isfinite(eps) || eps < 0.0f) return fail(SVDQ_STATUS_INVALID_VALUE, "eps must be finite and >= 0");
  if (!std::isfinite(residual_scale)) return fail(SVDQ_STATUS_INVALID_VALUE, "residual_scale must be finite");
  const bool has_y = y != nullptr, has_z = norm != SVDQ_NORM_NONE, mod = scale || shift;
  // (rows of an empty batch may be null, so they tell nothing of its parts)
  if (M > 0 && !has_y && !has_z) return fail(SVDQ_STATUS_INVALID_VALUE, "neither a block output nor a norm");
  if (M > 0 && !has_y && (gate || post_weight || post_norm != SVDQ_NORM_NONE))
    return fail(SVDQ_STATUS_INVALID_VALUE, "gate and post norm need a block output y");
  if (!has_z && (weight || mod || smooth || q8))
    return fail(SVDQ_STATUS_INVALID_VALUE, "weight, scale, shift, smooth and 8-bit output need a norm");
  if (post_weight && post_norm == SVDQ_NORM_NONE)
    return fail(SVDQ_STATUS_INVALID_VALUE, "post_weight needs a post norm");
  if (smooth && !q8) return fail(SVDQ_STATUS_INVALID_VALUE, "smooth needs the 8-bit output");
  if (M == 0) return ok();
  if (!x || (has_y && !h) || (has_z && !z) || (q8 && !z_scales))
    return fail(SVDQ_STATUS_INVALID_VALUE, "null x/h/z/z_scales");
  if ((gate && (gate_rows <= 0 || M % gate_rows != 0)) || (mod && (mod_rows <= 0 || M % mod_rows != 0)))
    return fail(SVDQ_STATUS_INVALID_VALUE, "gate rows %lld and modulation rows %lld must divide M=%lld",
                (long long)gate_rows, (long long)mod_rows, (long long)M);
  if (M == 1) x_stride = y_stride = h_stride = C;  // strides of one row are not read
  if (x_stride < C || (has_y && (y_stride < C || h_stride < C)) || (gate && gate_rows > 1 && gate_stride < C) ||
      (mod && mod_rows > 1 && mod_stride < C))
    return fail(SVDQ_STATUS_INVALID_VALUE, "a row stride is smaller than C=%lld", (long long)C);
  if (x_stride % 8 != 0 || (has_y && (y_stride % 8 != 0 || h_stride % 8 != 0)) ||
      (gate && gate_rows > 1 && gate_stride % 8 != 0) || (mod && mod_rows > 1 && mod_stride % 8 != 0))
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "row strides must be multiples of 8 elements");
  const int64_t far = 1ll << 37;  // 2^24 rows of 4 bytes stay below 2^63
  if (x_stride > far || (has_y && (y_stride > far || h_stride > far)) || (gate && gate_rows > 1 && gate_stride > far) ||
      (mod && mod_rows > 1 && mod_stride > far))
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "a row stride is above 2^37");
  for (const void* p : {x, y, post_weight, gate, weight, scale, shift, (const void*)smooth, (const void*)h,
                        (const void*)z, (const void*)z_scales})
    if (bad_ptr(p)) return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  const size_t e = stream_type == SVDQ_STREAM_FP32 ? 4 : 2, c = (size_t)C, m = (size_t)M;
  const size_t gs = gate_rows > 1 ? (size_t)gate_stride : 0, ms = mod_rows > 1 ? (size_t)mod_stride : 0;
  const Rows rx{x, (size_t)x_stride * e, c * e, m, "x"}, ry{y, (size_t)y_stride * 2, c * 2, m, "y"},
      rg{gate, gs * 2, c * 2, (size_t)(gate ? gate_rows : 0), "gate"},
      rsc{scale, ms * 2, c * 2, (size_t)(mod ? mod_rows : 0), "scale"},
      rsh{shift, ms * 2, c * 2, (size_t)(mod ? mod_rows : 0), "shift"}, rpw{post_weight, 0, c * 2, 1, "post_weight"},
      rw{weight, 0, c * 2, 1, "weight"}, rsm{smooth, 0, c * 4, 1, "smooth"},
      rh{has_y ? h : nullptr, (size_t)h_stride * e, c * e, m, "h"},
      rz{has_z ? z : nullptr, c * (q8 ? 1 : 2), c * (q8 ? 1 : 2), m, "z"},
      rzs{q8 ? z_scales : nullptr, 0, m * 4, 1, "z_scales"};
  // h may be x, and with it y, or a gate of M rows, where these are x too: a row's x,
  // y and gate are read before its h is written, scale and shift after it
  svdq_status s = SVDQ_STATUS_SUCCESS;
  if (has_y && unless_in_place(rh, rx).p == nullptr)
    s = check_rows(rh, {unless_in_place(rh, ry), unless_in_place(rh, rg), rsc, rsh, rpw, rw, rsm, rz, rzs});
  else
    s = check_rows(rh, {rx, ry, rg, rsc, rsh, rpw, rw, rsm, rz, rzs});
  if (s == SVDQ_STATUS_SUCCESS) s = check_rows(rz, {rx, ry, rg, rsc, rsh, rpw, rw, rsm, rzs});
  if (s == SVDQ_STATUS_SUCCESS) s = check_rows(rzs, {rx, ry, rg, rsc, rsh, rpw, rw, rsm});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  svdq::GateNormArgs a{};
  a.x = x;
  a.y = static_cast<const uint16_t*>(y);
  a.post_weight = static_cast<const uint16_t*>(post_weight);
  a.gate = static_cast<const uint16_t*>(gate);
  a.weight = static_cast<const uint16_t*>(weight);
  a.scale = static_cast<const uint16_t*>(scale);
  a.shift = static_cast<const uint16_t*>(shift);
  a.smooth = smooth;
  a.h = h;
  a.z = z;
  a.scales = q8 ? z_scales : nullptr;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.h_stride = h_stride;
  a.gate_stride = (int64_t)gs;
  a.mod_stride = (int64_t)ms;
  a.M = (int)M;
  a.C = (int)C;
  a.gate_every = gate ? (int)(M / gate_rows) : (int)M;
  a.mod_every = mod ? (int)(M / mod_rows) : (int)M;
  a.post = post_norm;
  a.norm = norm;
  a.x_fp32 = stream_type == SVDQ_STREAM_FP32;
  a.alpha = residual_scale;
  a.eps = eps;
  return launched(svdq::launch_gate_norm(a, static_cast<hipStream_t>(stream)), "gate norm");
}

svdq_status svdq_rope_axes_tables(const void* positions, int position_type, int64_t M, int64_t n_axes,
                                  const int64_t* axes, double theta, int spectrum, float* rope_cos, float* rope_sin,
                                  void* stream) {
  if (M < 0) return fail(SVDQ_STATUS_INVALID_VALUE, "bad dims M=%lld", (long long)M);
  if (!known_positions(position_type)) return fail(SVDQ_STATUS_INVALID_VALUE, "unknown position type %d", position_type);
  svdq::RopeAxes x{};
  svdq_status s = read_axes(n_axes, axes, theta, spectrum, x);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (M > kMaxRows) return fail(SVDQ_STATUS_NOT_SUPPORTED, "problem too large M=%lld", (long long)M);
  if (M == 0) return ok();
  if (!positions || !rope_cos || !rope_sin)
    return fail(SVDQ_STATUS_INVALID_VALUE, "null positions/rope_cos/rope_sin");
  if (bad_ptr(positions) || bad_ptr(rope_cos) || bad_ptr(rope_sin))
    return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  s = check_disjoint({{rope_cos, sz(M, x.half, 4), "rope_cos"}, {rope_sin, sz(M, x.half, 4), "rope_sin"}},
                     {{positions, sz(M, n_axes, 4), "positions"}});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  return launched(svdq::launch_rope_tables(positions, position_type == SVDQ_POSITIONS_INT32, x, M, rope_cos, rope_sin,
                                           static_cast<hipStream_t>(stream)), "rope tables");
}

svdq_status svdq_rope_axes(const void* q, int64_t q_stride, int64_t q_heads, const void* k, int64_t k_stride,
                           int64_t k_heads, int64_t head_dim, int64_t M, const void* positions, int position_type,
                           int64_t position_rows, int64_t n_axes, const int64_t* axes, double theta, int spectrum,
                           int layout, const void* q_norm, const void* k_norm, float eps, void* q_out,
                           int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (M < 0 || q_heads <= 0 || k_heads < 0 || head_dim <= 0)
    return fail(SVDQ_STATUS_INVALID_VALUE, "bad dims M=%lld q_heads=%lld k_heads=%lld head_dim=%lld", (long long)M,
                (long long)q_heads, (long long)k_heads, (long long)head_dim);
  if (head_dim % 8 != 0 || head_dim > 256)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "head_dim %lld (a multiple of 8, at most 256)", (long long)head_dim);
  if (M > kMaxRows || q_heads > 4096 || k_heads > 4096)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "problem too large M=%lld q_heads=%lld k_heads=%lld", (long long)M,
                (long long)q_heads, (long long)k_heads);
  if (!known_positions(position_type)) return fail(SVDQ_STATUS_INVALID_VALUE, "unknown position type %d", position_type);
  if (layout != SVDQ_ROPE_PAIRS && layout != SVDQ_ROPE_HALVES)
    return fail(SVDQ_STATUS_INVALID_VALUE, "unknown layout %d", layout);
  svdq::RopeAxes x{};
  svdq_status s = read_axes(n_axes, axes, theta, spectrum, x);
  if (s != SVDQ_STATUS_SUCCESS) return s;
  if (2 * x.half > head_dim)
    return fail(SVDQ_STATUS_INVALID_VALUE, "the axes take %d channels, a head has %lld", 2 * x.half, (long long)head_dim);
  if (layout == SVDQ_ROPE_HALVES && x.half % 4 != 0)
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "halves of %d channels (a multiple of 4)", x.half);
  if (!std::isfinite(eps) || eps < 0.0f) return fail(SVDQ_STATUS_INVALID_VALUE, "eps must be finite and >= 0");
  if (M == 0) return ok();
  const bool has_k = k_heads > 0;
  if (!q || !q_out || !positions || (has_k && (!k || !k_out)))
    return fail(SVDQ_STATUS_INVALID_VALUE, "null q/k/positions/q_out/k_out");
  if (has_k && (q_norm == nullptr) != (k_norm == nullptr))
    return fail(SVDQ_STATUS_INVALID_VALUE, "q_norm and k_norm go together");
  if (!has_k && k_norm) return fail(SVDQ_STATUS_INVALID_VALUE, "k_norm without k");
  if (position_rows <= 0 || M % position_rows != 0)
    return fail(SVDQ_STATUS_INVALID_VALUE, "position rows %lld must divide M=%lld", (long long)position_rows, (long long)M);
  const int64_t wq = q_heads * head_dim, wk = k_heads * head_dim;
  if (q_stride < wq || q_out_stride < wq || (has_k && (k_stride < wk || k_out_stride < wk)))
    return fail(SVDQ_STATUS_INVALID_VALUE, "a row stride is smaller than its heads");
  if (q_stride % 8 != 0 || q_out_stride % 8 != 0 || (has_k && (k_stride % 8 != 0 || k_out_stride % 8 != 0)))
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "row strides must be multiples of 8 elements");
  const int64_t far = 1ll << 38;
  if (q_stride > far || q_out_stride > far || (has_k && (k_stride > far || k_out_stride > far)))
    return fail(SVDQ_STATUS_NOT_SUPPORTED, "a row stride is above 2^38");
  for (const void* p : {q, k, positions, q_norm, k_norm, (const void*)q_out, (const void*)k_out})
    if (bad_ptr(p)) return fail(SVDQ_STATUS_INVALID_VALUE, "device pointers must be 16-byte aligned");
  const size_t m = (size_t)M, d = (size_t)head_dim;
  const Rows rq{q, (size_t)q_stride * 2, (size_t)wq * 2, m, "q"},
      rk{has_k ? k : nullptr, (size_t)k_stride * 2, (size_t)wk * 2, m, "k"},
      rp{positions, 0, (size_t)position_rows * (size_t)n_axes * 4, 1, "positions"}, rqn{q_norm, 0, d * 2, 1, "q_norm"},
      rkn{k_norm, 0, d * 2, 1, "k_norm"}, oq{q_out, (size_t)q_out_stride * 2, (size_t)wq * 2, m, "q_out"},
      ok_{has_k ? k_out : nullptr, (size_t)k_out_stride * 2, (size_t)wk * 2, m, "k_out"};
  s = check_rows(oq, {unless_in_place(oq, rq), rk, rp, rqn, rkn, ok_});
  if (s == SVDQ_STATUS_SUCCESS && has_k) s = check_rows(ok_, {rq, unless_in_place(ok_, rk), rp, rqn, rkn});
  if (s != SVDQ_STATUS_SUCCESS) return s;
  s = check_current_device();
  if (s != SVDQ_STATUS_SUCCESS) return s;
  svdq::RopeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(has_k ? k : nullptr);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(has_k ? k_out : nullptr);
  a.q_norm = static_cast<const uint16_t*>(q_norm);
  a.k_norm = static_cast<const uint16_t*>(k_norm);
  a.positions = positions;
  a.q_stride = q_stride;
  a.k_stride = has_k ? k_stride : 0;
  a.qo_stride = q_out_stride;
  a.ko_stride = has_k ? k_out_stride : 0;
  a.pos_rows = position_rows;
  a.M = (int)M;
  a.q_heads = (int)q_heads;
  a.k_heads = (int)k_heads;
  a.D = (int)head_dim;
  a.pos_int = position_type == SVDQ_POSITIONS_INT32;
  a.eps = eps;
  return launched(svdq::launch_rope_axes(a, x, layout == SVDQ_ROPE_HALVES, static_cast<hipStream_t>(stream)),
                  "rope axes");
}

}  // extern "C"
