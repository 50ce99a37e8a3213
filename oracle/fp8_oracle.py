"""CPU oracle of the 8-bit floating-point linear and the gated feed-forward block on it
(numpy, float64): e4m3 codes, one fp32 scale for a token's 128 channels and for 128 x 128
weights.  Shares no code with the HIP path.  Roundings that the definition names (the
fp32 scale, its reciprocal and their product, the bf16 x_hat, the codes) are made, no
others."""
from __future__ import annotations

import numpy as np

from .block_oracle import gelu_tanh
from .svdq_oracle import bf16_to_f64, f64_to_bf16

f32, f64 = np.float32, np.float64
BLOCK = 128


def _values():
    """The value of each of the 256 codes, float64 (NaN for 0x7F and 0xFF)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (c & 127) == 127 else v
        if c & 128:
            out[c] = -out[c]
    return out


VALUES = _values()


def decode(codes):
    return VALUES[np.asarray(codes, np.uint8)]


def encode(v):
    """The code nearest to v (finite, at most 464 in magnitude): by the borders between
    neighbouring values, ties to the even code."""
    v = np.asarray(v, f64)
    top = VALUES[:127]
    borders = (top[:-1] + top[1:]) / 2          # exact
    a = np.abs(v)
    low = np.searchsorted(borders, a, side="left")    # a on a border: the lower code
    high = np.searchsorted(borders, a, side="right")  # the upper one
    c = np.where(low % 2 == 0, low, high)
    return (c | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize(v):
    """v float64 [M, K] (fp32 values) -> (codes uint8 [M, K], scales fp32 [ceil(K / 128), M])."""
    v = np.asarray(v, f64)
    codes, scales = np.zeros(v.shape, np.uint8), []
    for k in range(0, v.shape[1], BLOCK):
        b = v[:, k:k + BLOCK]
        with np.errstate(all="ignore"):
            amax = np.abs(b).max(1).astype(f32)
            s = (amax * (f32(1) / f32(448))).astype(f32)
            inv = (f32(1) / s).astype(f32)
            dead = ~np.isfinite(inv) | ~np.isfinite(amax)
            t = (b.astype(f32) * inv[:, None]).astype(f32)
        codes[:, k:k + BLOCK] = np.where(dead[:, None], 0, encode(np.where(dead[:, None], 0.0, t)))
        scales.append(np.where(np.isfinite(amax), s, f32(np.nan)))
    return codes, np.array(scales, f32)


def quantize_act_fp8(x, smooth=None):
    """x float64 [M, K] (bf16 values), smooth fp32 [K] or None."""
    xh = np.asarray(x, f64)
    if smooth is not None:
        with np.errstate(all="ignore"):
            mu = (f32(1) / np.asarray(smooth, f32)).astype(f32)
            xh = bf16_to_f64(f64_to_bf16((xh.astype(f32) * mu[None, :]).astype(f32).astype(f64)))
    return quantize(xh)


def token_values(codes, scales):
    return decode(codes) * np.repeat(scales.astype(f64), BLOCK, 0)[:codes.shape[1]].T


def weight_values(codes, scales):
    N, K = codes.shape
    return decode(codes) * np.repeat(np.repeat(scales.astype(f64), BLOCK, 0), BLOCK, 1)[:N, :K]


def product(codes, scales, w_codes, w_scales, bias=None):
    """(the product with its bias, float64 [M, N]; the sum of its products' magnitudes)."""
    x, w = token_values(codes, scales), weight_values(w_codes, w_scales)
    y = x @ w.T
    return (y if bias is None else y + np.asarray(bias, f64)[None, :]), np.abs(x) @ np.abs(w).T


def fp8_gemm(codes, scales, w_codes, w_scales, bias=None, epilogue="none"):
    y = product(codes, scales, w_codes, w_scales, bias)[0]
    return gelu_tanh(y) if epilogue == "gelu_tanh" else y


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def fp8_gated_gemm(codes, scales, gate, up, gate_bias=None, up_bias=None, activation="silu"):
    """gate, up: (codes, scales)."""
    g, u = product(codes, scales, *gate, gate_bias)[0], product(codes, scales, *up, up_bias)[0]
    return (silu(g) if activation == "silu" else gelu_tanh(g)) * u


def pack_weights_fp8(w, smooth=None):
    """w float64 [N, K] -> (codes uint8 [N, K], scales fp32 [ceil(N / 128), ceil(K / 128)])."""
    w = np.asarray(w, f64) if smooth is None else np.asarray(w, f64) * np.asarray(smooth, f64)
    N, K = w.shape
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((-(-N // BLOCK), -(-K // BLOCK)), f32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[BLOCK * i:BLOCK * (i + 1), BLOCK * j:BLOCK * (j + 1)]
            s = f32(np.abs(w[at]).max() / 448)
            scales[i, j] = s
            if s > 0:
                codes[at] = encode(np.clip(w[at] / f64(s), -448, 448))
    return codes, scales
