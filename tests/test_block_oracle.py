"""Pins of the block operators' oracle (oracle/block_oracle.py) against something other
than itself: exact rationals, identities and hand-derived values."""
from fractions import Fraction

import numpy as np
import pytest

import oracle as O
import oracle.block_oracle as B


def _bf16(a):
    return O.bf16_to_f64(O.f64_to_bf16(np.asarray(a, np.float64)))


def test_token_scale_and_codes_by_hand():
    # max 127: s = 1, codes are the values, halves to even
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 3.0]])
    q, s = B.quantize_act_int8(x)
    assert s.tolist() == [1.0] and q.tolist() == [[127, 0, 2, 2, 0, -2, -126, 3]]
    q, s = B.quantize_act_int8(np.array([[0.0, 0.0], [np.inf, 1.0], [np.nan, 1.0], [-np.inf, 0.0]]))
    assert s[0] == 0 and np.isnan(s[1:]).all() and not q.any()
    # smoothing divides by a power of two: the same codes, another scale
    a, sa = B.quantize_act_int8(x, np.full(8, 4.0, np.float32))
    assert np.array_equal(a, B.quantize_act_int8(x)[0]) and sa[0] == 0.25


def test_quantizer_error_and_symmetry():
    g = np.random.default_rng(0)
    x = _bf16(g.standard_normal((20, 96)) * np.exp(g.standard_normal((20, 1))))
    q, s = B.quantize_act_int8(x)
    assert (np.abs(q).max(1) == 127).all()
    assert (np.abs(q * s[:, None].astype(float) - x) <= s[:, None] * 0.5 * (1 + 2.0 ** -15)).all()
    assert np.array_equal(B.quantize_act_int8(-x)[0], -q)


def test_gemm_against_rationals():
    g = np.random.default_rng(1)
    qx, qw = g.integers(-128, 128, (3, 70), dtype=np.int8), g.integers(-128, 128, (4, 70), dtype=np.int8)
    sx, sw = g.random(3).astype(np.float32), g.random(4).astype(np.float32)
    b = _bf16(g.standard_normal(4))
    y, _ = B.w8a8_gemm(qx, sx, qw, sw, b)
    for m in range(3):
        for n in range(4):
            acc = sum(int(a) * int(c) for a, c in zip(qx[m], qw[n]))
            want = Fraction(acc) * Fraction(float(sx[m])) * Fraction(float(sw[n])) + Fraction(float(b[n]))
            assert abs(float(want) - y[m, n]) <= 1e-12 * (1 + abs(float(want)))
    assert np.allclose(B.w8a8_gemm(qx, sx, qw, sw, b, "gelu_tanh")[0], O.gelu_tanh(y), rtol=0, atol=1e-12)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_identities(kind):
    g = np.random.default_rng(2)
    v = g.standard_normal((5, 64)) * 3 + 1
    n = B.unit_norm(v, kind, 0.0)
    assert np.allclose((n * n).mean(1), 1) and np.allclose(B.unit_norm(7 * v, kind, 0.0), n)
    if kind == "layer":
        assert np.allclose(n.mean(1), 0) and np.allclose(B.unit_norm(v + 5, kind, 0.0), n)
    h, z = B.gate_norm_modulate(v, v, gate=np.full((1, 64), 2.0), residual_scale=-2.0, norm=kind)
    assert not h.any() and not z.any()
    # the pieces one after another
    y, gate, sc, sh = (g.standard_normal(s) for s in ((6, 8), (3, 8), (2, 8), (2, 8)))
    x = g.standard_normal((6, 8))
    h, z = B.gate_norm_modulate(x, y, post_norm="rms", gate=gate, residual_scale=0.5, norm=kind, scale=sc, shift=sh)
    for m in range(6):
        u = y[m] / np.sqrt((y[m] ** 2).sum() / 8 + 1e-6)
        hm = 0.5 * x[m] + gate[m // 2] * u
        d = hm - (hm.sum() / 8 if kind == "layer" else 0)
        zm = d / np.sqrt((d ** 2).sum() / 8 + 1e-6) * (1 + sc[m // 3]) + sh[m // 3]
        assert np.allclose(h[m], hm) and np.allclose(z[m], zm)
    assert B.gate_norm_modulate(x, y, norm="none")[1] is None


@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("spectrum", ["axis", "shared"])
def test_rope_identities(layout, spectrum):
    g = np.random.default_rng(3)
    axes = (4, 2, 6)
    v = g.standard_normal((4, 3, 16))
    pos = g.integers(0, 50, (4, 3)).astype(float)
    kw = dict(axes=axes, spectrum=spectrum, layout=layout)
    out = B.rope_axes(v, pos, **kw)
    assert np.allclose((out ** 2).sum(-1), (v ** 2).sum(-1)) and np.array_equal(out[..., 12:], v[..., 12:])
    assert np.allclose(B.rope_axes(out, -pos, **kw), v) and np.array_equal(B.rope_axes(v, 0 * pos, **kw), v)
    # scores depend on position differences only
    k = g.standard_normal((4, 3, 16))
    a = (B.rope_axes(v, pos + 7, **kw) * B.rope_axes(k, pos * 0 + 7, **kw)).sum(-1)
    b = (out * B.rope_axes(k, pos * 0, **kw)).sum(-1)
    assert np.allclose(a, b)
    # one axis: both spectra agree
    one = dict(axes=(12,), layout=layout)
    assert np.allclose(B.rope_axes(v, pos[:, :1], spectrum="axis", **one), B.rope_axes(v, pos[:, :1], spectrum="shared", **one))


def test_rope_by_hand_and_against_the_qkv_oracle():
    t = B.rope_angles(np.array([[3.0, 5.0]]), (4, 2), theta=100.0)
    assert np.allclose(t, [[3.0, 3.0 / 10, 5.0 - 2 * np.pi]])
    t = B.rope_angles(np.array([[3.0, 5.0]]), (4, 2), theta=1000.0, spectrum="shared")
    assert np.allclose(t, [[3.0, 0.3, 0.05]])
    g = np.random.default_rng(4)
    v = g.standard_normal((5, 2, 128))
    pos = g.integers(0, 64, (5, 3)).astype(float)
    ang = B.rope_angles(pos, (16, 56, 56))
    want = O.rope_pairs(v.reshape(5, 256), 128, np.cos(ang), np.sin(ang)) if hasattr(O, "rope_pairs") else None
    if want is not None:
        assert np.allclose(B.rope_axes(v, pos, (16, 56, 56)).reshape(5, 256), want)


def test_rope_far_positions_keep_their_precision():
    """A position of 2^30 against the same angle from exact rational reduction."""
    t = B.rope_angles(np.array([[2.0 ** 30]]), (2,))
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    r = Fraction(2 ** 30) / (2 * pi)
    r -= round(r)
    assert abs(float(r * 2 * pi) - t[0, 0]) < 1e-8
