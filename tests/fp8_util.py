"""Helpers of the 8-bit floating-point linear's tests: values on both sides and the error
bounds that its arithmetic allows.

The matrix cores add products eight at a time (eight neighbours along K), cut off at
2^-13 of the power of two 2^r, r the largest sum of two codes' exponents in the group; the
groups, and blocks, are then added in fp32.  Random codes here take four neighbouring
exponents, so that a product's last bit, 2^-6 of its own exponent sum, is never below
the cut: a group's sum is exact, and a block's 16 groups pass through at most 16
additions, each of which is given a whole fp32 step (2 U, so that a truncating adder
passes).  The scale product, one fma per block and the joining of K-splits round by U
each.  For codes of any exponents cut_bound adds what the cut takes."""
from __future__ import annotations

import numpy as np

import oracle.fp8_oracle as F
from tests.block_util import U, bf16, dev


def dev_codes(c):
    import torch
    return dev(c).view(torch.float8_e4m3fn)


def host_codes(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def acts(M, K, seed):
    g = np.random.default_rng([seed, M, K])
    x = g.standard_normal((M, K))
    x[:, g.permutation(K)[:max(1, K // 100)]] *= 30
    return bf16(x), g


def _codes(g, rows, K):
    c = (g.integers(0, 2, (rows, K)) << 7) | (g.integers(6, 10, (rows, K)) << 3) | g.integers(0, 8, (rows, K))
    return np.where(g.random((rows, K)) < 0.05, 0, c).astype(np.uint8)


def tokens(M, K, seed):
    """Codes and scales of M tokens: scales that differ by powers of e."""
    g = np.random.default_rng([seed, M, K, 1])
    return _codes(g, M, K), (np.exp(g.standard_normal((-(-K // 128), M))) * 0.5).astype(np.float32)


def weights(N, K, seed):
    g = np.random.default_rng([seed, N, K, 2])
    return _codes(g, N, K), (np.exp(g.standard_normal((-(-N // 128), -(-K // 128)))) * 1e-2).astype(np.float32)


def product_bound(K, mags, y):
    """Of a product with K channels, the sum of its products' magnitudes and its value
    with the bias, for codes whose groups are exact."""
    return (2 * 16 + -(-K // 128) + 16 + 4) * U * mags + U * np.abs(y)


def cut_bound(codes, scales, w_codes, w_scales):
    """What the cut can take of a product: each of a group's products but the largest by less
    than 2^-13 of 2^r, r at most the sum of both sides' largest exponents."""
    def tops(c, s):
        e = np.maximum((c >> 3) & 15, 1).astype(int) - 7
        t = 2.0 ** e.reshape(c.shape[0], -1, 8).max(2)
        return t * np.repeat(s, 16, 1)[:, :t.shape[1]]
    wide = np.repeat(w_scales.astype(float), 128, 0)[:w_codes.shape[0]]
    return 7 * 2.0 ** -13 * tops(codes, scales.astype(float).T) @ tops(w_codes, wide).T


def act_bound(v, ev):
    """Of SiLU or GELU of v known up to ev: slopes stay below 1.13, the functions' own
    errors below 16 U |v| (tests of their tails are apart)."""
    return 1.15 * ev + 16 * U * np.abs(v)


def gated_bound(codes, scales, gate, up, gate_bias, up_bias, activation, cut=False):
    """(H, its bound) before the output rounding; cut: codes of any exponents."""
    K = codes.shape[1]
    g, mg = F.product(codes, scales, *gate, gate_bias)
    u, mu = F.product(codes, scales, *up, up_bias)
    eg, eu = product_bound(K, mg, g), product_bound(K, mu, u)
    if cut:
        eg, eu = eg + cut_bound(codes, scales, *gate), eu + cut_bound(codes, scales, *up)
    a = F.silu(g) if activation == "silu" else F.gelu_tanh(g)
    ea = act_bound(g, eg)
    h = a * u
    return h, np.abs(u) * ea + (np.abs(a) + ea) * eu + U * np.abs(h)
