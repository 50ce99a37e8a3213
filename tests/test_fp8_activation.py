"""The relative errors of the gated product's activations against the bounds that their
comments state (csrc/fp8.h, csrc/w8a8.h): the fp32 steps of the exponent on the CPU, and the
functions themselves on the GPU, to fp32 precision."""
import os
import re

import numpy as np
import pytest

import oracle.fp8_oracle as F
from tests.block_util import U, dev
from tests.fp8_util import dev_codes

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_diffusion_transformer_svdq_amd", "csrc")
f32, wide = np.float32, np.longdouble   # 64 bits of mantissa: a product of two fp32 values is exact


def _stated(name, var):
    """(a, b) of the bound (a |var| + b) 2^-24 in a header's comment."""
    text = re.sub(r"\s*\n//\s*", " ", open(os.path.join(CSRC, name)).read())
    m = re.search(r"relative error (?:stays )?below \(([\d.]*) ?\|%s\| \+ (\d+)\) 2\^-24" % var, text)
    assert m, name
    return float(m.group(1) or 1), float(m.group(2))


def _points(lo, hi, scale):
    """Arguments from lo to hi, dense just past the powers of two of scale x, where a
    product's rounding weighs most."""
    g = np.random.default_rng(5)
    p = 2.0 ** np.arange(-3, 8) / scale
    p = (p[:, None] * (1 + 0.02 * g.random(20000))).ravel()
    p = np.concatenate([p, g.uniform(lo, hi, 200000)])
    return np.unique(p[(p >= lo) & (p <= hi)].astype(f32))


# what follows the exponent: v_exp_f32 and v_rcp_f32 within a step (2 U), the sum and the
# last product rounded (U each)
REST = 2 + 2 + 1 + 1


def test_silu_exponent():
    a, b = _stated("fp8.h", "x")
    x = _points(1e-2, 87, 1.4427)
    t = (f32(1.442695041) * x).astype(f32)
    err = np.abs(t.astype(wide) * np.log(wide(2)) - x) / wide(U)   # of exp(-x), relative, in U
    assert b >= REST and (err <= a * x).all(), float((err / x).max())


def test_gelu_exponent():
    a, b = _stated("w8a8.h", "t")
    x = _points(1e-2, 10, 2.3022)
    c0, c1 = f32(2.302208198), f32(0.1029432397)
    sq = (x * x).astype(f32)
    s = (-(wide(c1) * sq.astype(wide)) - wide(c0)).astype(f32)          # one rounding, as the fma
    t = (x * s).astype(f32)
    w = x.astype(wide)
    exact = -2 * np.sqrt(2 / wide(np.pi)) * (w + wide("0.044715") * w ** 3) / np.log(wide(2))
    err = np.abs(t.astype(wide) - exact) * np.log(wide(2)) / wide(U)
    assert b >= REST and (err <= a * np.abs(exact)).all(), float((err / np.abs(exact)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [16, 30000])
def test_on_the_device(act, M):
    """Gates of any fp32 value: a token's scale times a code of 1 or -1.  U is the scale too,
    and the block's scale gives act(+-x) x to fp32 precision: the function's own error, the
    product's rounding and the scale's."""
    import bit_diffusion_transformer_svdq_amd as P
    top = 80 if act == "silu" else 9.9
    x = _points(1e-2, top, 1.4427 if act == "silu" else 2.3022)
    x = np.concatenate([[f32(44.3716926574707)], x])[:M] if M == 16 and act == "silu" else np.random.default_rng(M).permutation(x)[:M]
    x = x.astype(f32)
    codes = np.zeros((M, 128), np.uint8)
    codes[:, 9] = 0x38
    one = np.ones((1, 1), f32)
    up = np.zeros((128, 128), np.uint8)
    up[:, 9] = 0x38
    for sign in (1.0, -1.0):
        gate = np.zeros((128, 128), np.uint8)
        gate[:, 9] = F.encode(sign)
        _, s = P.fp8_gated_gemm(dev_codes(codes), dev(x[None]), dev_codes(gate), dev(one), dev_codes(up), dev(one),
                                activation=act, quantize="fp8")
        got = s.cpu().numpy()[0].astype(wide) / wide(f32(1) / f32(448))
        v = sign * x.astype(wide)
        if act == "silu":
            a, b = _stated("fp8.h", "x")
            e, arg = np.exp(-v), np.abs(v)
        else:
            a, b = _stated("w8a8.h", "t")
            t = -2 * np.sqrt(2 / wide(np.pi)) * (v + wide("0.044715") * v ** 3)
            e, arg = np.exp(t), np.abs(t) / np.log(wide(2))
        want = x.astype(wide) * x.astype(wide) / (1 + e)
        lim = 1.001 * (a * arg + b + 2) * wide(U)
        rel = np.abs(got / want - 1)
        assert (rel <= lim).all(), float((rel / lim).max())
