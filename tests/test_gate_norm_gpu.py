"""The gated residual norms (svdq_gate_norm_modulate) against the oracle.  Needs
an MI355X.  Bounds: tests/block_util.py."""
import numpy as np
import pytest

import oracle.block_oracle as B
from tests.block_util import HALF_BF16, U, bf16, check, dev, dev_bf16, gate_norm_bound, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _inputs(M, C, fp32, y, post, gate_rows, mod_rows, weight, seed):
    g = np.random.default_rng([seed, M, C])
    x = g.standard_normal((M, C)) * 2 + 0.5
    x[:, g.permutation(C)[:max(1, C // 100)]] *= 30
    p = dict(x=x.astype(np.float32).astype(np.float64) if fp32 else bf16(x))
    if y:
        p["y"] = bf16(g.standard_normal((M, C)) * 0.7 - 0.2)
        if gate_rows:
            p["gate"] = bf16(g.standard_normal((gate_rows, C)))
        if post != "none":
            p["post_norm"] = post
            if weight:
                p["post_weight"] = bf16(1 + 0.2 * g.standard_normal(C))
    if mod_rows:
        p["scale"], p["shift"] = bf16(0.4 * g.standard_normal((mod_rows, C))), bf16(0.4 * g.standard_normal((mod_rows, C)))
    if weight:
        p["weight"] = bf16(1 + 0.2 * g.standard_normal(C))
    return p, g


def _dev(p, fp32):
    d = {k: (dev_bf16(v) if isinstance(v, np.ndarray) else v) for k, v in p.items()}
    if fp32:
        d["x"] = dev(p["x"].astype(np.float32))
    return d


def _check(p, got, fp32, **kw):
    h, eh, z, ez = gate_norm_bound(**p, **kw)
    ref_h, ref_z = B.gate_norm_modulate(**p, **kw)
    if "y" in p:
        check(host(got[0]), ref_h, eh, U if fp32 else HALF_BF16)
    else:
        assert got[0] is None
    if ref_z is not None:
        check(host(got[1]), ref_z, ez)


SHAPES = [(1, 8), (1, 64), (3, 72), (5, 520), (4, 1536), (6, 2304), (2, 3072), (3, 4096), (2, 4104), (2, 8192), (2, 8200),
          (1, 16384), (2, 16392), (1, 32768), (2052, 512), (2050, 1032), (2049, 1544), (2053, 2056), (2060, 2568),
          (2056, 3072), (2052, 3592), (2051, 4096)]


@pytest.mark.parametrize("M,C", SHAPES)
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("kind,post", [("layer", "none"), ("rms", "rms"), ("rms", "layer"), ("layer", "rms")])
def test_block(M, C, fp32, kind, post):
    """Gated residual, both norms and modulation, every way a row is spread over waves."""
    import bit_diffusion_transformer_svdq_amd as P
    rows = M if M < 10 else (2 if M % 2 == 0 else 1)
    p, _ = _inputs(M, C, fp32, True, post, rows, rows, post == "rms", 1)
    got = P.gate_norm_modulate(**_dev(p, fp32), norm=kind, residual_scale=0.75)
    _check(p, got, fp32, norm=kind, residual_scale=0.75)


@pytest.mark.parametrize("kw", [dict(), dict(y=True), dict(y=True, gate_rows=1), dict(mod_rows=1), dict(weight=True),
                                dict(y=True, gate_rows=6, mod_rows=3), dict(y=True, gate_rows=2, mod_rows=6, weight=True)])
@pytest.mark.parametrize("norm", ["layer", "rms", "none"])
def test_parts(kw, norm):
    """Every part may be missing."""
    import bit_diffusion_transformer_svdq_amd as P
    a = dict(y=False, post="none", gate_rows=0, mod_rows=0, weight=False)
    a.update(kw)
    if norm == "none":
        a.update(mod_rows=0, weight=False, y=True)
    p, _ = _inputs(6, 136, False, seed=2, **a)
    got = P.gate_norm_modulate(**_dev(p, False), norm=norm)
    assert (got[1] is None) == (norm == "none")
    _check(p, got, False, norm=norm)


def test_only_scale_or_only_shift():
    import bit_diffusion_transformer_svdq_amd as P
    for drop in ("scale", "shift"):
        p, _ = _inputs(4, 264, True, True, "none", 1, 2, False, 3)
        p.pop(drop)
        _check(p, P.gate_norm_modulate(**_dev(p, True)), True)


@pytest.mark.parametrize("M", [7, 2100])
def test_strided_rows_and_update_in_place(M):
    """Chunks of one modulation row, rows of wider buffers, h written over x; what
    lies between the rows stays."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    C = 320
    p, g = _inputs(M, C, False, True, "none", M, M, False, 4)
    d = _dev(p, False)
    mod = torch.full((M, 3 * C + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    mod[:, :C], mod[:, C:2 * C], mod[:, 2 * C:3 * C] = d["gate"], d["scale"], d["shift"]
    xs = torch.full((M, C + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ys = torch.full((M, 2 * C), float("nan"), dtype=torch.bfloat16, device="cuda")
    xs[:, :C], ys[:, C:] = d["x"], d["y"]
    got = P.gate_norm_modulate(xs[:, :C], ys[:, C:], gate=mod[:, :C], scale=mod[:, C:2 * C], shift=mod[:, 2 * C:3 * C],
                               h_out=xs[:, :C])
    assert got[0].data_ptr() == xs.data_ptr() and bool((xs[:, C:] == 3).all())
    _check(p, got, False)


@pytest.mark.parametrize("M,C", [(1, 64), (3, 192), (5, 3072), (2, 4160), (3, 16384), (2, 32768), (2100, 576), (2049, 3072)])
@pytest.mark.parametrize("fp32,smooth,place", [(False, True, False), (True, False, False), (False, False, True)])
def test_int8_output(M, C, fp32, smooth, place):
    """Codes and scale of v = z / smooth: the scale within v's bound of max|v| / 127,
    each code within half a step of v."""
    import bit_diffusion_transformer_svdq_amd as P
    p, g = _inputs(M, C, fp32, True, "rms", 1, 1, True, 5)
    sm = np.exp(0.5 * g.standard_normal(C)).astype(np.float32) if smooth else None
    d = _dev(p, fp32)
    h, (q, s) = P.gate_norm_modulate(**d, quantize="int8", smooth=None if sm is None else dev(sm),
                                     h_out=d["x"] if place else None)
    hw, eh, z, ez = gate_norm_bound(**p)
    check(host(h), hw, eh, U if fp32 else HALF_BF16)
    if smooth:
        z, ez = z / sm, ez / sm
        ez = ez + 2 * U * np.abs(z)
    q, s = host(q), host(s)
    top, etop = np.abs(z).max(1), ez.max(1)
    assert (np.abs(s - top / 127) <= 1.02 * (etop / 127 + 2 * U * top)).all()
    assert (np.abs(q).max(1) == 127).all()
    assert (np.abs(q * s[:, None] - z) <= 1.001 * (0.5 * s[:, None] + ez + 256 * U * s[:, None])).all()


def test_int8_output_odd_rows():
    """A constant row (layer norm: zero), and rows with an infinity or NaN: codes 0
    with scale 0 or NaN, the others as without them."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    for M in (6, 2052):
        g = torch.Generator().manual_seed(M)
        x = torch.randn(M, 256, generator=g).cuda().bfloat16()
        x[1] = 3.0
        _, (q0, s0) = P.gate_norm_modulate(x, quantize="int8")
        assert float(s0[1]) == 0 and not bool(q0[1].any())
        y = x.clone()
        y[2, 5], y[4, 9] = float("inf"), float("nan")
        _, (q, s) = P.gate_norm_modulate(y, quantize="int8")
        bad = torch.tensor([2, 4], device="cuda")
        assert bool(s[bad].isnan().all()) and not bool(q[bad].any())
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])


def test_large_mean():
    """A mean a thousand times the deviation: the centered squares keep the variance."""
    import bit_diffusion_transformer_svdq_amd as P
    g = np.random.default_rng(6)
    p = dict(x=(1000 + g.standard_normal((5, 1024))).astype(np.float32).astype(np.float64))
    _check(p, P.gate_norm_modulate(dev(p["x"].astype(np.float32))), True)


def test_far_rows():
    """A stream whose last rows lie beyond 4 GiB of its start (row stride 2^28)."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    p, _ = _inputs(9, 256, False, True, "none", 1, 1, False, 7)
    d = _dev(p, False)
    buf = torch.zeros(8 * (1 << 28) + 256, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((9, 256), (1 << 28, 1))
    x.copy_(d["x"])
    d["x"] = x
    _check(p, P.gate_norm_modulate(**d, h_out=x), False)


def test_empty():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h, z = P.gate_norm_modulate(x, x)
    assert h.shape == (0, 64) and z.shape == (0, 64)


def test_most_rows():
    """2^24 rows on 4 waves each: more threads than one launch has, so a workgroup
    takes more than one row.  Every row as in a small call."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    M, C, B_ = 1 << 24, 2112, 4096
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 125 << 30:
        pytest.skip("needs 125 GiB of free device memory")
    small = torch.randn(B_, C, device="cuda").bfloat16()
    _, (want, ws) = P.gate_norm_modulate(small, norm="rms", quantize="int8")
    x = torch.empty(M, C, dtype=torch.bfloat16, device="cuda")
    x.view(-1, B_, C).copy_(small)
    _, (q, s) = P.gate_norm_modulate(x, norm="rms", quantize="int8")
    assert bool((s.view(-1, B_) == ws).all())
    q = q.view(-1, B_, C)
    for i in range(0, q.shape[0], 256):
        assert bool((q[i:i + 256] == want).all()), i
    del x, q, s
    torch.cuda.empty_cache()
