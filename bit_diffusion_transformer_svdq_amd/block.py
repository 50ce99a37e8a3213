"""The operators around the 4-bit linears of a transformer block: the 8-bit linear,
the gated residual norms and the rotary positions with several axes.

Like the rest of the binding this module only checks and marshals arguments
and allocates outputs; the arithmetic is in the library (include/svdq.h).  A call
runs on the current device's current stream, or on ``stream``: its outputs then
belong to that stream, and tensors given to it are kept for it if they are freed
meanwhile; ordering the two streams is the caller's part.  Tensors of another device are refused.

A block's pass, with the modulation vectors from ``awq_w4a16_gemm``::

    h, (q, s) = gate_norm_modulate(x, y, gate=gate, scale=scale, shift=shift, quantize="int8")
    qkv = w8a8_gemm(q, s, w_codes, w_scales, bias)
    q, k = rope_axes(qkv_q, qkv_k, positions, (16, 56, 56), q_norm=qn, k_norm=kn)
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _WS, _workspace
from ._lib import check, lib

_NORMS = {"none": 0, "layer": 1, "rms": 2}
_EPILOGUES = {"none": 0, "gelu_tanh": 1}
_SPECTRA = {"axis": 0, "shared": 1}
_LAYOUTS = {"pairs": 0, "halves": 1}
_NORM_OUTS = {None: 0, "int8": 1, "fp8": 3}
_BF16 = torch.bfloat16
_E4M3 = torch.float8_e4m3fn
_WS_COUNTERS = 1 << 20  # bytes of a workspace's arrival counters


def _choice(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: expected one of {sorted(table)}, got {value!r}") from None


def _device(t, stream, name):
    """The device index of a call's first tensor, which is the current device and the
    stream's (-1: an empty host tensor)."""
    idx = t.get_device()
    if idx < 0:
        if t.numel():
            raise ValueError(f"{name}: must be a device tensor")
        return idx
    here = _here()
    if idx != here or (stream is not None and stream.device_index != here):
        raise ValueError(f"{name}: the tensors, the stream and the current device (cuda:{here}) must agree")
    return idx


def _current_stream(idx):
    return torch.cuda.current_stream(idx).cuda_stream


# the handle of the current stream without a Stream object around it (2 us less
# per call), and the current device without a look at the initialization (a device
# tensor is in hand), where this torch has them
_raw_current = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_here = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _raw_stream(idx, stream):
    if stream is not None:
        return stream.cuda_stream
    return _raw_current(idx) if idx >= 0 else None


def _new(like, dtype, stream, *shape):
    """A contiguous tensor of this shape on the device of `like`, memory of `stream`."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(like, dtype, None, *shape)
    n = len(shape)
    strides = (1,) if n == 1 else (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)


def _new_like(t, stride, stream, *shape):
    """_new of t's own type and shape; empty_like is the quicker where t's rows are dense."""
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    return torch.empty_like(t) if stream is None and stride == width else _new(t, t.dtype, stream, *shape)


def _hold(stream, *tensors):
    """Memory of these tensors is not reused before what `stream` has been given is done."""
    for t in tensors:
        if t is not None and t.get_device() >= 0:
            t.record_stream(stream)


def _gemm_workspace(need, device, stream, given):
    """As the other calls' workspaces, except under capture: there every call gets
    memory of the graph's own, its arrival counters cleared by the graph, so that
    graphs captured on one stream share nothing."""
    if given is not None:
        return _workspace(need, device, stream, given)
    if stream is not None:
        with torch.cuda.stream(stream):
            return _gemm_workspace(need, device, None, None)
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty((need,), dtype=torch.uint8, device=device)
        ws[:_WS_COUNTERS].zero_()
        return ws.data_ptr(), need
    # (the current stream's, if it is large enough, without a Stream object: 2.5 us less per call)
    buf = _WS.get((device.index, _raw_current(device.index)))
    if buf is not None and buf.numel() >= need:
        return buf.data_ptr(), buf.numel()
    return _workspace(need, device, None, None)


def _refuse(t, dtype, shape, idx, name):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != idx:
        raise ValueError(f"{name}: must be on the device of the others, got {t.device}")
    raise ValueError(f"{name}: {'a row ' if len(shape) > 1 else ''}must be contiguous")


def _dense(t, dtype, shape, idx, name):
    """A contiguous tensor of exactly this type, shape and device -> its address."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == idx and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, shape, idx, name)


def _rows(t, dtype, shape, idx, name):
    """As _dense, but rows (dimension 0) may lie any distance apart -> (address, row stride)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == idx:
        strides = t.stride()
        if shape[0] > 1 and t.is_contiguous():
            return t.data_ptr(), strides[0]
        width = 1
        for d in range(len(shape) - 1, 0, -1):
            if strides[d] != width and shape[d] != 1:
                break
            width *= shape[d]
        else:
            return t.data_ptr(), strides[0] if shape[0] > 1 else width
    _refuse(t, dtype, shape, idx, name)


def _rows2(t, dtype, rows, width, idx, name):
    """_rows of a matrix, the common case, in one look at its strides."""
    if t.dtype is dtype and t.get_device() == idx and t.shape == (rows, width):
        stride, step = t.stride()
        if step == 1 or width == 1:
            return t.data_ptr(), stride if rows > 1 else width
    _refuse(t, dtype, (rows, width), idx, name)


def quantize_act_int8(x, smooth=None, out=None, stream=None):
    """Per-token 8-bit quantization: x bf16 [M, K], smooth fp32 [K] or None (x is
    divided by it) -> (act_codes int8 [M, K], act_scales fp32 [M])."""
    M, K = x.shape
    idx = _device(x, stream, "x")
    px = _dense(x, _BF16, (M, K), idx, "x")
    ps = None if smooth is None else _dense(smooth, torch.float32, (K,), idx, "smooth")
    if out is None:
        codes, scales = _new(x, torch.int8, stream, M, K), _new(x, torch.float32, stream, M)
        pc, pa = codes.data_ptr(), scales.data_ptr()
    else:
        codes, scales = out
        pc = _dense(codes, torch.int8, (M, K), idx, "act_codes")
        pa = _dense(scales, torch.float32, (M,), idx, "act_scales")
    check(lib().svdq_quantize_act_int8(px, ps, M, K, pc, pa, _raw_stream(idx, stream)), "svdq_quantize_act_int8")
    if stream is not None:
        _hold(stream, x, smooth, codes, scales)
    return codes, scales


def w8a8_gemm(act_codes, act_scales, w_codes, w_scales, bias=None, out=None, stream=None, epilogue="none",
              workspace=None):
    """8-bit linear: act_codes int8 [M, K], act_scales fp32 [M], w_codes int8 [N, K],
    w_scales fp32 [N], bias bf16 [N] or None -> Y bf16 [M, N].

    epilogue "gelu_tanh" applies GELU (tanh form) to y + b before the rounding.
    """
    M, K = act_codes.shape
    N = w_codes.shape[0]
    idx = _device(act_codes, stream, "act_codes")
    pa = _dense(act_codes, torch.int8, (M, K), idx, "act_codes")
    ps = _dense(act_scales, torch.float32, (M,), idx, "act_scales")
    pw = _dense(w_codes, torch.int8, (N, K), idx, "w_codes")
    pz = _dense(w_scales, torch.float32, (N,), idx, "w_scales")
    pb = None if bias is None else _dense(bias, _BF16, (N,), idx, "bias")
    epi = _choice(_EPILOGUES, epilogue, "epilogue")
    if out is None:
        y = _new(act_codes, _BF16, stream, M, N)
        py = y.data_ptr()
    else:
        y = out
        py = _dense(y, _BF16, (M, N), idx, "y")
    L = lib()
    need = L.svdq_w8a8_gemm_workspace_size(M, N, K)
    ws, wsb = (None, 0) if need == 0 and workspace is None else _gemm_workspace(
        need, act_codes.device, stream, workspace)
    check(L.svdq_w8a8_gemm(pa, ps, pw, pz, pb, M, N, K, epi, py, ws, wsb, _raw_stream(idx, stream)), "svdq_w8a8_gemm")
    if stream is not None:
        _hold(stream, act_codes, act_scales, w_codes, w_scales, bias, y, workspace)
    return y


def debug_set_w8a8_plan(tile: int = 0, splits: int = 0) -> None:
    """Test hook: w8a8_gemm's kernel and K-splits for later calls (0 = by shape)."""
    check(lib().svdq_debug_set_w8a8_plan(int(tile), int(splits)), "svdq_debug_set_w8a8_plan")


def gate_norm_modulate(x, y=None, post_norm="none", post_weight=None, gate=None, residual_scale=1.0, norm="layer",
                       weight=None, scale=None, shift=None, eps=1e-6, quantize=None, smooth=None, h_out=None,
                       out=None, stream=None):
    """The norms around a block, its gate and the residual scale in one pass:

        h = residual_scale * x + gate * post_norm(y) * post_weight
        z = norm(h) * weight * (1 + scale) + shift

    x bf16 or fp32 [M, C] (the residual stream), y bf16 [M, C] or None (h = x);
    norms "none", "layer" or "rms"; gate, scale, shift bf16 [B, C] with B dividing
    M (row m takes row m // (M // B)) or None; weights bf16 [C] or None.  Rows of
    x, y, gate, scale, shift and h may be strided (chunks of a projection's output).
    ``quantize="int8"`` gives z as the codes and token scales of w8a8_gemm,
    ``quantize="fp8"`` as the codes and block scales of fp8_gemm, divided by
    ``smooth`` (fp32 [C]) first.

    Returns (h, z): h of x's type, None without y (``h_out`` may be x); z bf16
    [M, C], or (int8 [M, C], fp32 [M]), or (float8_e4m3fn [M, C], fp32
    [ceil(C / 128), M]), or None for norm="none".
    """
    M, C = x.shape
    idx = _device(x, stream, "x")
    fp32 = x.dtype is torch.float32
    px, xs = _rows2(x, torch.float32 if fp32 else _BF16, M, C, idx, "x")
    post, kind = _choice(_NORMS, post_norm, "post_norm"), _choice(_NORMS, norm, "norm")
    if quantize not in (None, "int8", "fp8"):
        raise ValueError(f"quantize: expected None, 'int8' or 'fp8', got {quantize!r}")
    out_type = _NORM_OUTS[quantize]
    py = ph = ppw = pg = pw = psc = psh = psm = pz = pzs = None
    ys = hs = gr = gs = mr = ms = 0
    h = z = None
    if y is not None:
        py, ys = _rows2(y, _BF16, M, C, idx, "y")
        if h_out is None:
            h = _new_like(x, xs, stream, M, C)
            ph, hs = h.data_ptr(), C
        else:
            h = h_out
            ph, hs = _rows2(h, x.dtype, M, C, idx, "h")
    elif h_out is not None:
        raise ValueError("h_out: there is no h without y")
    if post_weight is not None:
        ppw = _dense(post_weight, _BF16, (C,), idx, "post_weight")
    if gate is not None:
        gr = gate.shape[0]
        pg, gs = _rows2(gate, _BF16, gr, C, idx, "gate")
    if weight is not None:
        pw = _dense(weight, _BF16, (C,), idx, "weight")
    if scale is not None:
        mr = scale.shape[0]
        psc, ms = _rows2(scale, _BF16, mr, C, idx, "scale")
    if shift is not None:
        if scale is None:
            mr = shift.shape[0]
        psh, shs = _rows2(shift, _BF16, mr, C, idx, "shift")
        if scale is not None and shs != ms:
            raise ValueError("scale and shift: the row strides differ")
        ms = shs
    if smooth is not None:
        psm = _dense(smooth, torch.float32, (C,), idx, "smooth")
    if kind:
        if quantize is None:
            if out is None:
                z = _new(x, _BF16, stream, M, C) if fp32 else _new_like(x, xs, stream, M, C)
                pz = z.data_ptr()
            else:
                z = out
                pz = _dense(z, _BF16, (M, C), idx, "z")
        else:
            codes, shape = (torch.int8, (M,)) if quantize == "int8" else (_E4M3, (-(-C // 128), M))
            if out is None:
                z = _new(x, codes, stream, M, C), _new(x, torch.float32, stream, *shape)
                pz, pzs = z[0].data_ptr(), z[1].data_ptr()
            else:
                z = (out[0], out[1])
                pz = _dense(z[0], codes, (M, C), idx, "z codes")
                pzs = _dense(z[1], torch.float32, shape, idx, "z scales")
    elif out is not None:
        raise ValueError("out: there is no z with norm='none'")
    check(lib().svdq_gate_norm_modulate(
        px, int(fp32), xs, py, ys, post, ppw, pg, gr, gs, residual_scale, kind, pw, psc, psh, mr, ms, eps, M, C,
        ph, hs, out_type, psm, pz, pzs, _raw_stream(idx, stream)), "svdq_gate_norm_modulate")
    if stream is not None:
        _hold(stream, x, y, post_weight, gate, weight, scale, shift, smooth, h, *(z if isinstance(z, tuple) else (z,)))
    return h, z


_MAX_ANGLES = 128  # angles of a head: half the axes' channels


def _axes_array(axes):
    a = (ctypes.c_int64 * len(axes))(*axes)
    if a[:] != list(axes):
        raise ValueError(f"axes: widths do not fit 64 bits: {tuple(axes)}")
    return a


def _positions(t, idx, n_axes):
    """positions fp32 or int32 [P, n_axes] -> (address, type code, P)."""
    if t.dtype is torch.float32:
        code = 0
    elif t.dtype is torch.int32:
        code = 1
    else:
        raise TypeError(f"positions: expected torch.float32 or torch.int32, got {t.dtype}")
    P = t.shape[0]
    return _dense(t, t.dtype, (P, n_axes), idx, "positions"), code, P


def rope_axes_tables(positions, axes, theta=10000.0, spectrum="axis", out=None, stream=None):
    """Cosines and sines of positions fp32 or int32 [M, len(axes)] -> (cos, sin), fp32
    [M, R/2], R = sum(axes): with R = 128 the tables of w4a4_gemm_qkv_norm_rope.

    axes: channels each axis turns.  spectrum "axis": each axis's rates fall from 1
    to about 1/theta over its own width; "shared": one series over all R channels,
    of which each axis owns a section."""
    idx = _device(positions, stream, "positions")
    pp, code, M = _positions(positions, idx, len(axes))
    ax = _axes_array(axes)
    half = sum(ax) // 2
    if out is None:
        if not 0 < half <= _MAX_ANGLES:
            half = 0  # the library refuses these axes: they ask for no memory first
        cos, sin = (_new(positions, torch.float32, stream, M, half) for _ in range(2))
    else:
        cos, sin = out
        _dense(cos, torch.float32, (M, half), idx, "cos")
        _dense(sin, torch.float32, (M, half), idx, "sin")
    check(lib().svdq_rope_axes_tables(pp, code, M, len(axes), ax, theta,
                                      _choice(_SPECTRA, spectrum, "spectrum"), cos.data_ptr(), sin.data_ptr(),
                                      _raw_stream(idx, stream)), "svdq_rope_axes_tables")
    if stream is not None:
        _hold(stream, positions, cos, sin)
    return cos, sin


def rope_axes(q, k, positions, axes, theta=10000.0, spectrum="axis", layout="pairs", q_norm=None, k_norm=None,
              eps=1e-6, out=None, stream=None):
    """Turns q bf16 [M, Hq, D] and k bf16 [M, Hk, D] (or None) by positions fp32 or int32
    [P, len(axes)], P dividing M (token m reads row m % P), after an optional RMSNorm
    per head (q_norm, k_norm bf16 [D]).  Tokens may be strided (the thirds of a QKV
    output); ``out=(q, k)`` turns in place.  axes and spectrum as for
    rope_axes_tables; layout "pairs" turns channels (2i, 2i+1), "halves" (i, i + R/2).
    Returns (q_out, k_out)."""
    M, Hq, D = q.shape
    idx = _device(q, stream, "q")
    pq, qs = _rows(q, _BF16, (M, Hq, D), idx, "q")
    pk = pko = None
    Hk = ks = kos = 0
    if k is not None:
        Hk = k.shape[1]
        pk, ks = _rows(k, _BF16, (M, Hk, D), idx, "k")
    if out is None:
        qo = _new_like(q, qs, stream, M, Hq, D)
        pqo, qos, ko = qo.data_ptr(), Hq * D, None
        if k is not None:
            ko = _new_like(k, ks, stream, M, Hk, D)
            pko, kos = ko.data_ptr(), Hk * D
    else:
        qo, ko = out
        if (ko is None) != (k is None):
            raise ValueError("out: one output for q and one for k")
        pqo, qos = _rows(qo, _BF16, (M, Hq, D), idx, "q_out")
        if k is not None:
            pko, kos = _rows(ko, _BF16, (M, Hk, D), idx, "k_out")
    pp, code, P = _positions(positions, idx, len(axes))
    pqn = None if q_norm is None else _dense(q_norm, _BF16, (D,), idx, "q_norm")
    pkn = None if k_norm is None else _dense(k_norm, _BF16, (D,), idx, "k_norm")
    check(lib().svdq_rope_axes(
        pq, qs, Hq, pk, ks, Hk, D, M, pp, code, P, len(axes), _axes_array(axes), theta,
        _choice(_SPECTRA, spectrum, "spectrum"), _choice(_LAYOUTS, layout, "layout"), pqn, pkn, eps, pqo, qos, pko,
        kos, _raw_stream(idx, stream)), "svdq_rope_axes")
    if stream is not None:
        _hold(stream, q, k, positions, q_norm, k_norm, qo, ko)
    return qo, ko


def pack_weights_int8(w_bf16: np.ndarray, smooth: np.ndarray | None = None) -> dict:
    """Host packer of the 8-bit linear: W bf16 bits [N, K], smooth fp32 [K] or None ->
    w_codes int8 [N, K], w_scales fp32 [N]."""
    w = np.ascontiguousarray(w_bf16, dtype=np.uint16)
    N, K = w.shape
    lam = None if smooth is None else np.ascontiguousarray(smooth, dtype=np.float32)
    if lam is not None and lam.shape != (K,):
        raise ValueError(f"smooth: expected shape ({K},), got {lam.shape}")
    codes = np.empty((N, K), dtype=np.int8)
    scales = np.empty((N,), dtype=np.float32)
    vp = ctypes.c_void_p
    check(lib().svdq_pack_weights_int8(w.ctypes.data_as(vp), None if lam is None else lam.ctypes.data_as(vp), N, K,
                                       codes.ctypes.data_as(vp), scales.ctypes.data_as(vp)),
          "svdq_pack_weights_int8")
    return {"w_codes": codes, "w_scales": scales}
