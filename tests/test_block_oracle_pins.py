"""The block operators' oracle against the fused QKV operator's, which was written apart
from it."""
import numpy as np
import pytest

import oracle as O
import oracle.block_oracle as B


@pytest.mark.parametrize("axes,D", [((16, 56, 56), 128), ((64,), 64), ((8, 24), 32)])
@pytest.mark.parametrize("spectrum", ["axis", "shared"])
def test_pairs_are_turned_as_the_qkv_oracle_turns_them(axes, D, spectrum):
    g = np.random.default_rng([4, D])
    v = g.standard_normal((5, 2, D))
    pos = g.integers(-64, 64, (5, len(axes))).astype(float)
    t = B.rope_angles(pos, axes, spectrum=spectrum)
    want = O.rope_pairs(v.reshape(5, 2 * D), D, np.cos(t), np.sin(t)).reshape(v.shape)
    assert np.allclose(B.rope_axes(v, pos, axes, spectrum=spectrum), want, rtol=0, atol=1e-13)


def test_head_norm_is_that_of_the_qkv_oracle():
    g = np.random.default_rng(5)
    v = g.standard_normal((5, 2, 64))
    w = O.f64_to_bf16(1 + 0.1 * g.standard_normal(64))
    pos = g.integers(0, 64, (5, 2)).astype(float)
    t = B.rope_angles(pos, (24, 40))
    n = O.rms_norm_heads(v.reshape(5, 128), 64, w, 1e-6)
    want = O.rope_pairs(n, 64, np.cos(t), np.sin(t)).reshape(v.shape)
    assert np.allclose(B.rope_axes(v, pos, (24, 40), norm_weight=O.bf16_to_f64(w)), want, rtol=0, atol=1e-12)
