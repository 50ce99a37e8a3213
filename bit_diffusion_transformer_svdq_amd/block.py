"""The operators around the 4-bit linears of a transformer block: the 8-bit linear,
the gated residual norms and the rotary positions with several axes.

Like the rest of the binding this module only checks and marshals arguments
and allocates outputs; the arithmetic is in the library (include/svdq.h).  A call
runs on the current device's current stream, or on ``stream``; tensors of
another device are refused.  A block's pass, with the modulation vectors from
``awq_w4a16_gemm``::

    h, (q, s) = gate_norm_modulate(x, y, gate=gate, scale=scale, shift=shift, quantize="int8")
    qkv = w8a8_gemm(q, s, w_codes, w_scales, bias)
    q, k = rope_axes(qkv_q, qkv_k, positions, (16, 56, 56), q_norm=qn, k_norm=kn)
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._lib import check, lib

_NORMS = {"none": 0, "layer": 1, "rms": 2}
_EPILOGUES = {"none": 0, "gelu_tanh": 1}
_SPECTRA = {"axis": 0, "shared": 1}
_LAYOUTS = {"pairs": 0, "halves": 1}
_BF16 = torch.bfloat16


def _choice(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: expected one of {sorted(table)}, got {value!r}") from None


def _device(t, stream, name):
    """The device of a call's first tensor: the stream's, or the current one."""
    dev = t.device
    if t.numel() and dev.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor")
    if dev.type == "cuda":
        here = torch.cuda.current_device()
        if dev.index != here or (stream is not None and stream.device_index != here):
            raise ValueError(f"{name}: the tensors, the stream and the current device (cuda:{here}) must agree")
    return dev


def _raw_stream(dev, stream):
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream(dev).cuda_stream if dev.type == "cuda" else None


def _dense(t, dtype, shape, dev, name):
    """A contiguous tensor of exactly this type, shape and device -> its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name}: must be on {dev}, got {t.device}")
    return t.data_ptr()


def _rows(t, dtype, shape, dev, name):
    """As _dense, but rows (dimension 0) may lie any distance apart -> (address, row stride)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: must be on {dev}, got {t.device}")
    width = 1
    strides = t.stride()
    for d in range(len(shape) - 1, 0, -1):
        if strides[d] != width and shape[d] != 1 and shape[0]:
            raise ValueError(f"{name}: a row must be contiguous")
        width *= shape[d]
    return t.data_ptr(), strides[0] if shape[0] > 1 else width


def quantize_act_int8(x, smooth=None, out=None, stream=None):
    """Per-token 8-bit quantization: x bf16 [M, K], smooth fp32 [K] or None (x is
    divided by it) -> (act_codes int8 [M, K], act_scales fp32 [M])."""
    M, K = x.shape
    dev = _device(x, stream, "x")
    px = _dense(x, _BF16, (M, K), dev, "x")
    ps = None if smooth is None else _dense(smooth, torch.float32, (K,), dev, "smooth")
    if out is None:
        codes = torch.empty((M, K), dtype=torch.int8, device=dev)
        scales = torch.empty((M,), dtype=torch.float32, device=dev)
        pc, pa = codes.data_ptr(), scales.data_ptr()
    else:
        codes, scales = out
        pc = _dense(codes, torch.int8, (M, K), dev, "act_codes")
        pa = _dense(scales, torch.float32, (M,), dev, "act_scales")
    check(lib().svdq_quantize_act_int8(px, ps, M, K, pc, pa, _raw_stream(dev, stream)), "svdq_quantize_act_int8")
    return codes, scales


def w8a8_gemm(act_codes, act_scales, w_codes, w_scales, bias=None, out=None, stream=None, epilogue="none",
              workspace=None):
    """8-bit linear: act_codes int8 [M, K], act_scales fp32 [M], w_codes int8 [N, K],
    w_scales fp32 [N], bias bf16 [N] or None -> Y bf16 [M, N].

    epilogue "gelu_tanh" applies GELU (tanh form) to y + b before the rounding.
    """
    from . import _workspace
    M, K = act_codes.shape
    N = w_codes.shape[0]
    dev = _device(act_codes, stream, "act_codes")
    pa = _dense(act_codes, torch.int8, (M, K), dev, "act_codes")
    ps = _dense(act_scales, torch.float32, (M,), dev, "act_scales")
    pw = _dense(w_codes, torch.int8, (N, K), dev, "w_codes")
    pz = _dense(w_scales, torch.float32, (N,), dev, "w_scales")
    pb = None if bias is None else _dense(bias, _BF16, (N,), dev, "bias")
    epi = _choice(_EPILOGUES, epilogue, "epilogue")
    if out is None:
        y = torch.empty((M, N), dtype=_BF16, device=dev)
        py = y.data_ptr()
    else:
        y = out
        py = _dense(y, _BF16, (M, N), dev, "y")
    L = lib()
    need = L.svdq_w8a8_gemm_workspace_size(M, N, K)
    ws, wsb = (None, 0) if need == 0 and workspace is None else _workspace(need, dev, stream, workspace)
    check(L.svdq_w8a8_gemm(pa, ps, pw, pz, pb, M, N, K, epi, py, ws, wsb, _raw_stream(dev, stream)), "svdq_w8a8_gemm")
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
    divided by ``smooth`` (fp32 [C]) first.

    Returns (h, z): h of x's type, None without y (``h_out`` may be x); z bf16
    [M, C], or (int8 [M, C], fp32 [M]), or None for norm="none".
    """
    M, C = x.shape
    dev = _device(x, stream, "x")
    fp32 = x.dtype is torch.float32
    px, xs = _rows(x, torch.float32 if fp32 else _BF16, (M, C), dev, "x")
    post, kind = _choice(_NORMS, post_norm, "post_norm"), _choice(_NORMS, norm, "norm")
    if quantize not in (None, "int8"):
        raise ValueError(f"quantize: expected None or 'int8', got {quantize!r}")
    py = ph = ppw = pg = pw = psc = psh = psm = pz = pzs = None
    ys = hs = gr = gs = mr = ms = 0
    h = z = None
    if y is not None:
        py, ys = _rows(y, _BF16, (M, C), dev, "y")
        h = torch.empty((M, C), dtype=x.dtype, device=dev) if h_out is None else h_out
        ph, hs = _rows(h, x.dtype, (M, C), dev, "h")
    elif h_out is not None:
        raise ValueError("h_out: there is no h without y")
    if post_weight is not None:
        ppw = _dense(post_weight, _BF16, (C,), dev, "post_weight")
    if gate is not None:
        gr = gate.shape[0]
        pg, gs = _rows(gate, _BF16, (gr, C), dev, "gate")
    if weight is not None:
        pw = _dense(weight, _BF16, (C,), dev, "weight")
    if scale is not None:
        mr = scale.shape[0]
        psc, ms = _rows(scale, _BF16, (mr, C), dev, "scale")
    if shift is not None:
        if scale is None:
            mr = shift.shape[0]
        psh, shs = _rows(shift, _BF16, (mr, C), dev, "shift")
        if scale is not None and shs != ms:
            raise ValueError("scale and shift: the row strides differ")
        ms = shs
    if smooth is not None:
        psm = _dense(smooth, torch.float32, (C,), dev, "smooth")
    if kind:
        if quantize is None:
            z = torch.empty((M, C), dtype=_BF16, device=dev) if out is None else out
            pz = z.data_ptr() if out is None else _dense(z, _BF16, (M, C), dev, "z")
        else:
            if out is None:
                z = (torch.empty((M, C), dtype=torch.int8, device=dev),
                     torch.empty((M,), dtype=torch.float32, device=dev))
                pz, pzs = z[0].data_ptr(), z[1].data_ptr()
            else:
                z = (out[0], out[1])
                pz = _dense(z[0], torch.int8, (M, C), dev, "z codes")
                pzs = _dense(z[1], torch.float32, (M,), dev, "z scales")
    elif out is not None:
        raise ValueError("out: there is no z with norm='none'")
    check(lib().svdq_gate_norm_modulate(
        px, int(fp32), xs, py, ys, post, ppw, pg, gr, gs, residual_scale, kind, pw, psc, psh, mr, ms, eps, M, C,
        ph, hs, int(quantize is not None), psm, pz, pzs, _raw_stream(dev, stream)), "svdq_gate_norm_modulate")
    return h, z


def _axes_array(axes):
    return (ctypes.c_int64 * len(axes))(*axes)


def _positions(t, dev, n_axes):
    """positions fp32 or int32 [P, n_axes] -> (address, type code, P)."""
    if t.dtype is torch.float32:
        code = 0
    elif t.dtype is torch.int32:
        code = 1
    else:
        raise TypeError(f"positions: expected torch.float32 or torch.int32, got {t.dtype}")
    P = t.shape[0]
    return _dense(t, t.dtype, (P, n_axes), dev, "positions"), code, P


def rope_axes_tables(positions, axes, theta=10000.0, spectrum="axis", out=None, stream=None):
    """Cosines and sines of positions fp32 or int32 [M, len(axes)] -> (cos, sin), fp32
    [M, R/2], R = sum(axes): with R = 128 the tables of w4a4_gemm_qkv_norm_rope.

    axes: channels each axis turns.  spectrum "axis": each axis's rates fall from 1
    to about 1/theta over its own width; "shared": one series over all R channels,
    of which each axis owns a section."""
    dev = _device(positions, stream, "positions")
    pp, code, M = _positions(positions, dev, len(axes))
    half = sum(axes) // 2
    if out is None:
        cos, sin = (torch.empty((M, half), dtype=torch.float32, device=dev) for _ in range(2))
    else:
        cos, sin = out
    pc = _dense(cos, torch.float32, (M, half), dev, "cos")
    ps = _dense(sin, torch.float32, (M, half), dev, "sin")
    check(lib().svdq_rope_axes_tables(pp, code, M, len(axes), _axes_array(axes), theta,
                                      _choice(_SPECTRA, spectrum, "spectrum"), pc, ps, _raw_stream(dev, stream)),
          "svdq_rope_axes_tables")
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
    dev = _device(q, stream, "q")
    pq, qs = _rows(q, _BF16, (M, Hq, D), dev, "q")
    pk = pko = None
    Hk = ks = kos = 0
    if k is not None:
        Hk = k.shape[1]
        pk, ks = _rows(k, _BF16, (M, Hk, D), dev, "k")
    if out is None:
        qo = torch.empty((M, Hq, D), dtype=_BF16, device=dev)
        ko = None if k is None else torch.empty((M, Hk, D), dtype=_BF16, device=dev)
    else:
        qo, ko = out
        if (ko is None) != (k is None):
            raise ValueError("out: one output for q and one for k")
    pqo, qos = _rows(qo, _BF16, (M, Hq, D), dev, "q_out")
    if k is not None:
        pko, kos = _rows(ko, _BF16, (M, Hk, D), dev, "k_out")
    pp, code, P = _positions(positions, dev, len(axes))
    pqn = None if q_norm is None else _dense(q_norm, _BF16, (D,), dev, "q_norm")
    pkn = None if k_norm is None else _dense(k_norm, _BF16, (D,), dev, "k_norm")
    check(lib().svdq_rope_axes(
        pq, qs, Hq, pk, ks, Hk, D, M, pp, code, P, len(axes), _axes_array(axes), theta,
        _choice(_SPECTRA, spectrum, "spectrum"), _choice(_LAYOUTS, layout, "layout"), pqn, pkn, eps, pqo, qos, pko,
        kos, _raw_stream(dev, stream)), "svdq_rope_axes")
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
