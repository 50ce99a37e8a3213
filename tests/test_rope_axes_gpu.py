"""Rotary positions with several axes (svdq_rope_axes_tables, svdq_rope_axes)
against the oracle.  Needs an MI355X.

Tables: two roundings of the double product (below 2^-52 of the angle each), sine and
cosine in double (below 2^-45), one rounding to fp32.
The turn: that error times |a| + |b|, three fp32 roundings, one to bf16."""
import numpy as np
import pytest

import oracle.block_oracle as B
from tests.block_util import U, bf16, check, dev, dev_bf16, host, norm_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _table_bound(pos, axes):
    # the fastest rate is 1 radian per unit
    return 1.01 * U + 2 * np.pi * 2 ** -51 * np.abs(pos).max()


def _pos(g, P, n, kind):
    if kind == "far":
        return g.integers(-2 ** 24, 2 ** 24, (P, n)).astype(np.float32)
    if kind == "int":
        return g.integers(-2 ** 31, 2 ** 31 - 1, (P, n)).astype(np.int32)
    if kind == "fraction":
        return (g.random((P, n)) * 100 - 50).astype(np.float32)
    return g.integers(0, 64, (P, n)).astype(np.float32)


@pytest.mark.parametrize("axes", [(16, 56, 56), (128,), (2,), (4, 2, 6), (44, 42, 42), (64, 64, 64, 64), (2,) * 8])
@pytest.mark.parametrize("P,kind", [(1, "grid"), (7, "far"), (257, "fraction"), (4608, "grid"), (33, "int")])
@pytest.mark.parametrize("spectrum", ["axis", "shared"])
def test_tables(axes, P, kind, spectrum):
    import bit_diffusion_transformer_svdq_amd as K
    pos = _pos(np.random.default_rng([1, P, len(axes)]), P, len(axes), kind)
    c, s = K.rope_axes_tables(dev(pos), axes, theta=10000.0, spectrum=spectrum)
    t = B.rope_angles(pos, axes, 10000.0, spectrum)
    e = _table_bound(pos, axes)
    assert c.shape == s.shape == (P, sum(axes) // 2)
    assert np.abs(host(c) - np.cos(t)).max() <= e and np.abs(host(s) - np.sin(t)).max() <= e


def test_positions_that_are_not_finite():
    """Their axis's channels become NaN; other axes and tokens are as without them."""
    import torch
    import bit_diffusion_transformer_svdq_amd as K
    g = np.random.default_rng(8)
    pos = _pos(g, 9, 2, "fraction")
    bad = pos.copy()
    bad[1, 0], bad[4, 1], bad[6, 0] = np.nan, np.inf, -np.inf
    axes = (16, 24)
    q = dev_bf16(bf16(g.standard_normal((9, 3, 48))))
    for t, b in zip((*K.rope_axes_tables(dev(pos), axes), K.rope_axes(q, None, dev(pos), axes)[0]),
                    (*K.rope_axes_tables(dev(bad), axes), K.rope_axes(q, None, dev(bad), axes)[0])):
        w = 2 if t.dim() == 3 else 1
        lost = torch.zeros_like(t, dtype=torch.bool)
        for m, lo, hi in ((1, 0, 8), (6, 0, 8), (4, 8, 20)):
            lost[m, ..., w * lo:w * hi] = True
        assert bool(b[lost].isnan().all()) and torch.equal(b[~lost], t[~lost])


def _check_turn(got, v, w, pos, axes, theta, spectrum, layout, eps=1e-6):
    n, en = (np.asarray(v), np.zeros_like(v)) if w is None else norm_bound(v, np.zeros_like(v), "rms", eps)
    if w is not None:
        n, en = n * w, en * np.abs(w) + 2 * U * np.abs(n * w)
    want = B.rope_axes(v, pos, axes, theta, spectrum, layout, w, eps)
    R = sum(axes)
    mate = np.zeros_like(n)
    emate = np.zeros_like(n)
    i = np.arange(R)
    j = i ^ 1 if layout == "pairs" else (i + R // 2) % R
    mate[..., :R], emate[..., :R] = n[..., j], en[..., j]
    et = _table_bound(pos, axes)
    err = en + emate + (et + 3 * U) * (np.abs(n) + np.abs(mate))
    check(got, want, err)


CASES = [  # M, P, Hq, Hk, D, axes, layout
    (1, 1, 1, 1, 128, (16, 56, 56), "pairs"), (3, 3, 24, 24, 128, (16, 56, 56), "pairs"), (5, 5, 3, 1, 64, (32, 32), "halves"),
    (4, 2, 16, 2, 128, (44, 42, 42), "halves"), (6, 1, 5, 5, 72, (24, 24, 24), "halves"), (7, 7, 4, 2, 72, (10, 14), "pairs"),
    (9, 3, 8, 0, 80, (40, 40), "halves"), (2, 2, 2, 1, 256, (128, 64, 64), "halves"), (2, 2, 3, 3, 256, (100, 20), "pairs"),
    (11, 11, 40, 8, 96, (8, 16, 24), "halves"), (5, 5, 7, 7, 8, (2, 2, 2), "pairs"), (5, 5, 9, 9, 8, (4, 4), "halves"),
    (3, 3, 64, 64, 24, (16,), "halves"), (1030, 515, 6, 2, 128, (16, 56, 56), "pairs"), (4100, 4100, 2, 1, 64, (16, 24, 24), "halves"),
    (8200, 4100, 3, 1, 40, (20, 12), "halves"), (2100, 2100, 24, 24, 128, (44, 42, 42), "halves")]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("norm", [False, True])
def test_turn(case, norm):
    import bit_diffusion_transformer_svdq_amd as K
    M, P, Hq, Hk, D, axes, layout = case
    g = np.random.default_rng([2, M, Hq, D])
    q, k = bf16(1.5 * g.standard_normal((M, Hq, D))), bf16(1.5 * g.standard_normal((M, Hk, D)))
    qn, kn = (bf16(1 + 0.2 * g.standard_normal(D)) for _ in range(2))
    pos = _pos(g, P, len(axes), ["grid", "fraction", "far", "int"][M % 4])
    spectrum = "shared" if M % 2 else "axis"
    qo, ko = K.rope_axes(dev_bf16(q), dev_bf16(k) if Hk else None, dev(pos), axes, theta=5000.0, spectrum=spectrum,
                         layout=layout, q_norm=dev_bf16(qn) if norm else None,
                         k_norm=dev_bf16(kn) if norm and Hk else None)
    _check_turn(host(qo), q, qn if norm else None, pos, axes, 5000.0, spectrum, layout)
    if Hk:
        _check_turn(host(ko), k, kn if norm else None, pos, axes, 5000.0, spectrum, layout)
    else:
        assert ko is None


@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("M", [3, 1500])
def test_in_place_on_a_fused_projection(M, layout):
    """Q and K thirds of one QKV buffer turned in place: V and the padding stay, and
    the values are those of the call out of place."""
    import torch
    import bit_diffusion_transformer_svdq_amd as K
    Hq, Hk, D, axes = 6, 2, 128, (16, 56, 56)
    wide = (Hq + 2 * Hk) * D + 64
    g = torch.Generator().manual_seed(M)
    buf = torch.randn(M, wide, generator=g).cuda().bfloat16()
    pos = torch.randint(0, 64, (M, 3), generator=g).int().cuda()
    qn, kn = (1 + 0.1 * torch.randn(2, D, generator=g)).cuda().bfloat16()
    q, k = buf[:, :Hq * D].unflatten(1, (Hq, D)), buf[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    keep = buf.clone()
    want = K.rope_axes(q, k, pos, axes, layout=layout, q_norm=qn, k_norm=kn)
    assert torch.equal(buf, keep)
    got = K.rope_axes(q, k, pos, axes, layout=layout, q_norm=qn, k_norm=kn, out=(q, k))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(buf[:, (Hq + Hk) * D:], keep[:, (Hq + Hk) * D:])


def test_tables_feed_the_fused_qkv_projection():
    """rope_axes on the plain projection's output gives what the fused QKV epilogue
    gives with the same positions' tables, up to the projection's own rounding
    to bf16 in between (HALF_BF16 of each channel, turned and normed)."""
    import torch
    import bit_diffusion_transformer_svdq_amd as K
    from tests.gpu_util import bf16_bits, custom_case, to_dev, to_dev_bf16
    import oracle as O
    M, Kd, heads, axes = 96, 256, 2, (16, 56, 56)
    d, lam, p = custom_case(M, Kd, 3 * heads * 128, 16, seed=5)
    g = np.random.default_rng(3)
    pos = dev(g.integers(0, 64, (M, 3)).astype(np.float32))
    qn, kn = dev_bf16(bf16(1 + 0.1 * g.standard_normal(128))), dev_bf16(bf16(1 + 0.1 * g.standard_normal(128)))
    c, s, la = K.quantize_act_lora_down(to_dev_bf16(d["x"]), to_dev(np.asarray(lam, np.float32)), to_dev_bf16(p["lora_down"]))
    args = (c, s, to_dev(p["w_codes"]), to_dev_bf16(p["w_scales"]), la, to_dev_bf16(p["lora_up"]), to_dev_bf16(d["bias"]))
    cos, sin = K.rope_axes_tables(pos, axes)
    fused = K.w4a4_gemm_qkv_norm_rope(*args, qn, kn, cos, sin)
    qkv = K.w4a4_gemm_lora_up(*args)
    E = heads * 128
    q, k = K.rope_axes(qkv[:, :E].unflatten(1, (heads, 128)), qkv[:, E:2 * E].unflatten(1, (heads, 128)), pos, axes,
                       q_norm=qn, k_norm=kn)
    for i, t in enumerate((q, k)):
        a, b = host(fused[:, i * E:(i + 1) * E]), host(t.flatten(1))
        # rounding of the projection: 2^-8 of the two channels of a pair (and as much
        # through the norm), rounding of either output: 2^-8 of it
        pair = np.hypot(a.reshape(M, -1, 2)[..., 0], a.reshape(M, -1, 2)[..., 1]).repeat(2, -1).reshape(a.shape)
        assert (np.abs(a - b) <= 2.0 ** -8 * (3 * pair * np.sqrt(2) + 2 * np.abs(a)) + 1e-6).all()
    assert torch.equal(qkv[:, 2 * E:], fused[:, 2 * E:])
    assert O is not None and bf16_bits is not None


def test_far_rows_and_empty():
    """Tokens beyond 4 GiB of the buffer's start; no tokens at all."""
    import torch
    import bit_diffusion_transformer_svdq_amd as K
    g = np.random.default_rng(9)
    q = bf16(g.standard_normal((9, 2, 64)))
    buf = torch.zeros(8 * (1 << 28) + 128, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((9, 2, 64), (1 << 28, 64, 1))
    t.copy_(dev_bf16(q))
    pos = g.integers(0, 50, (9, 2)).astype(np.float32)
    got, _ = K.rope_axes(t, None, dev(pos), (32, 32), out=(t, None))
    _check_turn(host(got), q, None, pos, (32, 32), 10000.0, "axis", "pairs")
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    qo, ko = K.rope_axes(e, e, torch.empty((0, 2), device="cuda"), (32, 32))
    assert qo.shape == ko.shape == (0, 2, 64)
