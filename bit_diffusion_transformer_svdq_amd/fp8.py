"""The 8-bit floating-point linear (e4m3 codes, an fp32 scale for a token's 128 channels
and for 128 x 128 weights) and the gated feed-forward block on it.

As block.py, this module only checks and marshals arguments and allocates outputs;
streams, devices and workspaces are handled as there.  A block's feed-forward part::

    h, (q, s) = gate_norm_modulate(x, y, gate=gate, scale=scale, shift=shift, quantize="fp8", smooth=sm)
    q, s = fp8_gated_gemm(q, s, wg, wg_scales, wu, wu_scales, quantize="fp8", smooth=sm_down)
    y = fp8_gemm(q, s, wd, wd_scales, bias)

Codes are float8_e4m3fn tensors; scales of activations are [ceil(K / 128), M], one row
per block, so that ``codes[a:b], scales[:, a:b]`` are those of the tokens a to b.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._lib import check, lib
from .block import (_BF16, _E4M3, _EPILOGUES, _choice, _dense, _device, _gemm_workspace, _hold, _new, _raw_stream,
                    _rows2)

_ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


def _blocks(n):
    return -(-n // 128)


def _coded(like, M, K, out, stream, idx, name):
    """The codes and scales that a call writes, given or new -> them, their addresses and
    the scales' row stride."""
    if out is None:
        codes, scales = _new(like, _E4M3, stream, M, K), _new(like, torch.float32, stream, _blocks(K), M)
        return codes, scales, codes.data_ptr(), scales.data_ptr(), M
    codes, scales = out
    pc = _dense(codes, _E4M3, (M, K), idx, name + "_codes")
    ps, stride = _rows2(scales, torch.float32, _blocks(K), M, idx, name + "_scales")
    return codes, scales, pc, ps, stride


def _weights(codes, scales, N, K, idx, name):
    return (_dense(codes, _E4M3, (N, K), idx, name + "_codes"),
            _dense(scales, torch.float32, (_blocks(N), _blocks(K)), idx, name + "_scales"))


def quantize_act_fp8(x, smooth=None, out=None, stream=None):
    """Block quantization: x bf16 [M, K], smooth fp32 [K] or None (x is divided by it) ->
    (act_codes float8_e4m3fn [M, K], act_scales fp32 [ceil(K / 128), M])."""
    M, K = x.shape
    idx = _device(x, stream, "x")
    px = _dense(x, _BF16, (M, K), idx, "x")
    psm = None if smooth is None else _dense(smooth, torch.float32, (K,), idx, "smooth")
    codes, scales, pc, ps, stride = _coded(x, M, K, out, stream, idx, "act")
    check(lib().svdq_quantize_act_fp8(px, psm, M, K, pc, ps, stride, _raw_stream(idx, stream)), "svdq_quantize_act_fp8")
    if stream is not None:
        _hold(stream, x, smooth, codes, scales)
    return codes, scales


def fp8_gemm(act_codes, act_scales, w_codes, w_scales, bias=None, out=None, stream=None, epilogue="none",
             workspace=None):
    """8-bit floating-point linear: act_codes float8_e4m3fn [M, K], act_scales fp32
    [ceil(K / 128), M] (rows may be strided), w_codes float8_e4m3fn [N, K], w_scales fp32
    [ceil(N / 128), ceil(K / 128)], bias bf16 [N] or None -> Y bf16 [M, N].

    epilogue "gelu_tanh" applies GELU (tanh form) to y + b before the rounding.
    """
    M, K = act_codes.shape
    N = w_codes.shape[0]
    idx = _device(act_codes, stream, "act_codes")
    pa = _dense(act_codes, _E4M3, (M, K), idx, "act_codes")
    ps, stride = _rows2(act_scales, torch.float32, _blocks(K), M, idx, "act_scales")
    pw, pz = _weights(w_codes, w_scales, N, K, idx, "w")
    pb = None if bias is None else _dense(bias, _BF16, (N,), idx, "bias")
    epi = _choice(_EPILOGUES, epilogue, "epilogue")
    if out is None:
        y = _new(act_codes, _BF16, stream, M, N)
        py = y.data_ptr()
    else:
        y = out
        py = _dense(y, _BF16, (M, N), idx, "y")
    L = lib()
    need = L.svdq_fp8_gemm_workspace_size(M, N, K)
    ws, wsb = (None, 0) if need == 0 and workspace is None else _gemm_workspace(
        need, act_codes.device, stream, workspace)
    check(L.svdq_fp8_gemm(pa, ps, stride, pw, pz, pb, M, N, K, epi, py, ws, wsb, _raw_stream(idx, stream)),
          "svdq_fp8_gemm")
    if stream is not None:
        _hold(stream, act_codes, act_scales, w_codes, w_scales, bias, y, workspace)
    return y


def fp8_gated_gemm(act_codes, act_scales, gate_codes, gate_scales, up_codes, up_scales, gate_bias=None, up_bias=None,
                   activation="silu", quantize=None, smooth=None, out=None, stream=None, workspace=None):
    """Both projections of a gated feed-forward block, its activation and the product in
    one kernel: h = act(x Wg^T + bg) * (x Wu^T + bu).

    act_codes and act_scales as for fp8_gemm; gate_codes, up_codes float8_e4m3fn [F, K],
    their scales fp32 [ceil(F / 128), ceil(K / 128)], biases bf16 [F] or None; activation
    "silu" or "gelu_tanh" (tanh form).  Returns h bf16 [M, F], or with
    ``quantize="fp8"`` its codes and scales as fp8_gemm reads them, divided by ``smooth``
    (fp32 [F]) first."""
    M, K = act_codes.shape
    F = gate_codes.shape[0]
    idx = _device(act_codes, stream, "act_codes")
    pa = _dense(act_codes, _E4M3, (M, K), idx, "act_codes")
    ps, stride = _rows2(act_scales, torch.float32, _blocks(K), M, idx, "act_scales")
    pg, pgs = _weights(gate_codes, gate_scales, F, K, idx, "gate")
    pu, pus = _weights(up_codes, up_scales, F, K, idx, "up")
    pbg = None if gate_bias is None else _dense(gate_bias, _BF16, (F,), idx, "gate_bias")
    pbu = None if up_bias is None else _dense(up_bias, _BF16, (F,), idx, "up_bias")
    psm = None if smooth is None else _dense(smooth, torch.float32, (F,), idx, "smooth")
    if quantize not in (None, "fp8"):
        raise ValueError(f"quantize: expected None or 'fp8', got {quantize!r}")
    act, kind = _choice(_ACTIVATIONS, activation, "activation"), int(quantize is not None)
    pos, os = None, 0
    if kind:
        h, scales, po, pos, os = _coded(act_codes, M, F, out, stream, idx, "out")
    elif out is None:
        h, scales = _new(act_codes, _BF16, stream, M, F), None
        po = h.data_ptr()
    else:
        h, scales = out, None
        po = _dense(h, _BF16, (M, F), idx, "out")
    L = lib()
    need = L.svdq_fp8_gated_gemm_workspace_size(M, F, K, kind)
    ws, wsb = (None, 0) if need == 0 and workspace is None else _gemm_workspace(
        need, act_codes.device, stream, workspace)
    check(L.svdq_fp8_gated_gemm(pa, ps, stride, pg, pgs, pu, pus, pbg, pbu, M, F, K, act, kind, psm, po, pos, os, ws, wsb,
                                _raw_stream(idx, stream)), "svdq_fp8_gated_gemm")
    if stream is not None:
        _hold(stream, act_codes, act_scales, gate_codes, gate_scales, up_codes, up_scales, gate_bias, up_bias, smooth, h,
              scales, workspace)
    return (h, scales) if kind else h


def gated_ffn_fp8(x, gate: dict, up: dict, down: dict, activation="silu", out=None, stream=None):
    """A gated feed-forward block on one stream: x bf16 [M, K] is quantized, both
    projections and the activation run as fp8_gated_gemm, whose codes the
    down-projection reads -> y bf16 [M, N].

    ``gate``, ``up`` and ``down`` hold the packed layers as device tensors: w_codes,
    w_scales, bias (or None), and in ``gate`` and ``down`` smooth (or None; gate's is that
    of the input both projections share)."""
    q, s = quantize_act_fp8(x, gate["smooth"], stream=stream)
    q, s = fp8_gated_gemm(q, s, gate["w_codes"], gate["w_scales"], up["w_codes"], up["w_scales"], gate["bias"], up["bias"],
                          activation=activation, quantize="fp8", smooth=down["smooth"], stream=stream)
    return fp8_gemm(q, s, down["w_codes"], down["w_scales"], down["bias"], out=out, stream=stream)


def debug_set_fp8_plan(tile: int = 0, splits: int = 0) -> None:
    """Test hook: the fp8 products' kernel and K-splits for later calls (0 = by shape)."""
    check(lib().svdq_debug_set_fp8_plan(int(tile), int(splits)), "svdq_debug_set_fp8_plan")


def pack_weights_fp8(w_bf16: np.ndarray, smooth: np.ndarray | None = None) -> dict:
    """Host packer of the 8-bit floating-point linear: W bf16 bits [N, K], smooth fp32 [K] or
    None -> w_codes uint8 [N, K] (e4m3 bits: a torch view of them as float8_e4m3fn is what the
    calls take), w_scales fp32 [ceil(N / 128), ceil(K / 128)]."""
    w = np.ascontiguousarray(w_bf16, dtype=np.uint16)
    N, K = w.shape
    lam = None if smooth is None else np.ascontiguousarray(smooth, dtype=np.float32)
    if lam is not None and lam.shape != (K,):
        raise ValueError(f"smooth: expected shape ({K},), got {lam.shape}")
    codes = np.empty((N, K), dtype=np.uint8)
    scales = np.empty((_blocks(N), _blocks(K)), dtype=np.float32)
    vp = ctypes.c_void_p
    check(lib().svdq_pack_weights_fp8(w.ctypes.data_as(vp), None if lam is None else lam.ctypes.data_as(vp), N, K,
                                      codes.ctypes.data_as(vp), scales.ctypes.data_as(vp)),
          "svdq_pack_weights_fp8")
    return {"w_codes": codes, "w_scales": scales}
