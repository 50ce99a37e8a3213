"""CPU oracle of the block operators (numpy, float64): the 8-bit linear, the gated
residual norms, the rotary positions with several axes.  Inputs are float64 or
float32 arrays of the values the device tensors hold; shares no code with the
HIP path.  Roundings that a definition names (the fp32 token scale and its
reciprocal, the bf16 x_hat) are made, no others."""
from __future__ import annotations

import numpy as np

from .svdq_oracle import bf16_to_f64, f64_to_bf16

f32, f64 = np.float32, np.float64


def token_scales(x_hat):
    """(s fp32 [M], fl32(1/s) fp32 [M]; 0 where the row's codes are 0) of x_hat [M, K]."""
    with np.errstate(all="ignore"):
        amax = np.abs(x_hat).max(1).astype(f32)  # a NaN stays one
        s = (amax / f32(127)).astype(f32)
        inv = (f32(1) / s).astype(f32)
    inv = np.where(np.isfinite(inv), inv, f32(0)).astype(f32)
    bad = ~np.isfinite(amax)
    return np.where(bad, f32(np.nan), s).astype(f32), np.where(bad, f32(0), inv).astype(f32)


def quantize_act_int8(x, smooth=None):
    """x float64 [M, K] (bf16 values), smooth fp32 [K] -> codes int8 [M, K], scales fp32 [M]."""
    with np.errstate(all="ignore"):
        xh = np.asarray(x, f64)
        if smooth is not None:
            mu = (f32(1) / np.asarray(smooth, f32)).astype(f32)
            xh = bf16_to_f64(f64_to_bf16((xh.astype(f32) * mu[None, :]).astype(f32).astype(f64)))
        s, inv = token_scales(xh)
        t = np.rint(xh * inv.astype(f64)[:, None])
        q = np.where(inv[:, None] == 0, 0.0, t)
    return q.astype(np.int8), s


def gelu_tanh(v):
    return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))


def w8a8_gemm(codes, s_x, w_codes, s_w, bias=None, epilogue="none"):
    """(Y float64 [M, N], the product part before the bias)."""
    acc = codes.astype(f64) @ w_codes.astype(f64).T  # exact below 2^53
    p = acc * s_x.astype(f64)[:, None] * s_w.astype(f64)[None, :]
    y = p if bias is None else p + np.asarray(bias, f64)[None, :]
    return (gelu_tanh(y) if epilogue == "gelu_tanh" else y), p


def unit_norm(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def _spread(v, M):
    v = np.asarray(v, f64)
    return np.repeat(v, M // v.shape[0], 0)


def gate_norm_modulate(x, y=None, post_norm="none", post_weight=None, gate=None, residual_scale=1.0, norm="layer",
                       weight=None, scale=None, shift=None, eps=1e-6):
    """(h, z) float64 [M, C]; h = x without y, z None for norm "none"."""
    h = np.asarray(x, f64)
    M = h.shape[0]
    if y is not None:
        u = np.asarray(y, f64)
        if post_norm != "none":
            u = unit_norm(u, post_norm, eps)
            if post_weight is not None:
                u = u * np.asarray(post_weight, f64)
        h = residual_scale * h + (u if gate is None else _spread(gate, M) * u)
    if norm == "none":
        return h, None
    z = unit_norm(h, norm, eps)
    if weight is not None:
        z = z * np.asarray(weight, f64)
    if scale is not None:
        z = z * (1 + _spread(scale, M))
    if shift is not None:
        z = z + _spread(shift, M)
    return h, z


def rope_angles(positions, axes, theta=10000.0, spectrum="axis"):
    """float64 [P, R/2], reduced by whole turns."""
    pos, R = np.asarray(positions, np.longdouble), sum(axes)
    cols, i = [], 0
    for a, d in enumerate(axes):
        for j in range(d // 2):
            e = np.longdouble(2 * j) / d if spectrum == "axis" else np.longdouble(2 * i) / R
            rev = pos[:, a] * np.exp(-e * np.log(np.longdouble(theta))) / (2 * np.longdouble("3.14159265358979323846264338"))
            cols.append(((rev - np.rint(rev)) * 2 * np.longdouble("3.14159265358979323846264338")).astype(f64))
            i += 1
    return np.stack(cols, 1)


def rope_axes(v, positions, axes, theta=10000.0, spectrum="axis", layout="pairs", norm_weight=None, eps=1e-6):
    """v float64 [M, H, D] -> turned float64 [M, H, D]; positions [P, n], M % P == 0."""
    v = np.asarray(v, f64)
    if norm_weight is not None:
        v = unit_norm(v, "rms", eps) * np.asarray(norm_weight, f64)
    t = rope_angles(positions, axes, theta, spectrum)
    t = np.tile(t, (v.shape[0] // t.shape[0], 1))[:, None, :]
    c, s, half = np.cos(t), np.sin(t), t.shape[2]
    out = v.copy()
    if layout == "pairs":
        a, b = v[..., 0:2 * half:2], v[..., 1:2 * half:2]
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = a * c - b * s, a * s + b * c
    else:
        a, b = v[..., :half], v[..., half:2 * half]
        out[..., :half], out[..., half:2 * half] = a * c - b * s, a * s + b * c
    return out
