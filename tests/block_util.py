"""Helpers of the block operators' tests: values on both sides, and the error bounds
that fp32 arithmetic and one final rounding allow.

U is the unit roundoff of fp32 (2^-24), HALF_BF16 that of bf16 (2^-8).  Bounds are
first order in U; SLACK covers the second order."""
from __future__ import annotations

import numpy as np

import oracle as O

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
SLACK = 1.02
# additions one partial sum passes through: at most 8 channels of 8 vectors in a
# lane, 6 steps across the wave, 16 waves; fma and the final products on top
ADDS = 64 + 6 + 16 + 4


def bf16(a):
    """float64 values rounded to bf16 (as float64)."""
    return O.bf16_to_f64(O.f64_to_bf16(np.asarray(a, np.float64)))


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def dev_bf16(a):
    import torch
    return None if a is None else dev(np.asarray(a, np.float32), torch.bfloat16)  # exact: bf16 values


def host(t):
    return t.detach().double().cpu().numpy()


def norm_bound(v, ev, kind, eps):
    """(unit norm of v, bound of its error) for v known up to ev elementwise."""
    if kind == "layer":
        d = v - v.mean(-1, keepdims=True)
        ed = ev + ev.mean(-1, keepdims=True) + ADDS * U * np.abs(v).mean(-1, keepdims=True) + 2 * U * (np.abs(v) + np.abs(d))
    else:
        d, ed = v, ev
    ss = (d * d).mean(-1, keepdims=True) + eps
    e_ss = 2 * (np.abs(d) * ed).mean(-1, keepdims=True) + ADDS * U * ss
    r = 1 / np.sqrt(ss)
    er = r * (e_ss / (2 * ss) + 4 * U)
    n = d * r
    return n, ed * r + np.abs(d) * er + 2 * U * np.abs(n)


def gate_norm_bound(x, y=None, post_norm="none", post_weight=None, gate=None, residual_scale=1.0, norm="layer",
                    weight=None, scale=None, shift=None, eps=1e-6):
    """(h, its bound, z, its bound) before the output rounding."""
    M = x.shape[0]
    h, eh = np.asarray(x, np.float64), np.zeros_like(x, dtype=np.float64)
    if y is not None:
        u, eu = np.asarray(y, np.float64), 0.0
        if post_norm != "none":
            u, eu = norm_bound(u, np.zeros_like(u), post_norm, eps)
            if post_weight is not None:
                u, eu = u * post_weight, eu * np.abs(post_weight)
            eu = eu + 2 * U * np.abs(u)
        g = 1.0 if gate is None else np.repeat(gate, M // gate.shape[0], 0)
        a = np.float64(np.float32(residual_scale))
        eh = np.abs(g) * eu + U * np.abs(a * h) + 2 * U * np.abs(a * h + g * u)
        h = a * h + g * u
    if norm == "none":
        return h, eh, None, None
    z, ez = norm_bound(h, eh, norm, eps)
    if weight is not None:
        z, ez = z * weight, ez * np.abs(weight)
    if scale is not None:
        sc = np.repeat(scale, M // scale.shape[0], 0)
        z, ez = z * (1 + sc), ez * np.abs(1 + sc) + 2 * U * np.abs(z) * (1 + np.abs(sc))
    ez = ez + 2 * U * np.abs(z)
    if shift is not None:
        sh = np.repeat(shift, M // shift.shape[0], 0)
        z = z + sh
        ez = ez + U * np.abs(z)
    return h, eh, z, ez


def check(got, want, err, half=HALF_BF16):
    """|got - want| within the arithmetic's bound plus one rounding of the result."""
    lim = SLACK * (err + half * (np.abs(want) + err)) + 1e-38
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], lim[bad][:4])
