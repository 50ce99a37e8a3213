"""What the block operators' contract says about memory and sizes, checked without a
GPU: every refusal comes before any HIP call, on pointers that are never read."""
import ctypes

import pytest

from bit_diffusion_transformer_svdq_amd._lib import INVALID_VALUE, NO_DEVICE, NOT_SUPPORTED, SUCCESS, lib
from tests.test_block_abi_host import NORM, ROPE, P, _call, _gpu_visible

# a bf16 stream of four rows, updated in place, with bf16 output
PLACE = dict(h=P(1), otype=0, smooth=None, zs=None, z=P(10))


@pytest.mark.parametrize("kw", [
    dict(gate=P(1), gr=2, gs=128),                      # row m reads gate row m / 2, which another row's update writes
    dict(scale=P(1), mr=2, ms=128), dict(shift=P(1), mr=2, ms=128),
    dict(scale=P(1), mr=4, ms=128), dict(shift=P(1), mr=4, ms=128),   # read after the row's h is written
    dict(scale=P(1), shift=P(1), mr=4, ms=128),
    dict(gate=P(1), gr=1, gs=0), dict(w=P(1)), dict(pw=P(1)), dict(z=P(1)),
    dict(y=P(1), ys=256), dict(h=P(8), hs=128, z=P(1)), dict(h=P(8), z=P(8))])
def test_an_update_in_place_shares_its_rows_with_nothing_else(kw):
    """h may be x itself; what a row reads after its h is written, or another row reads,
    lies elsewhere."""
    assert _call("svdq_gate_norm_modulate", NORM, dict(PLACE, **kw)) == INVALID_VALUE


@pytest.mark.skipif(_gpu_visible(), reason="checks the no-GPU path")
@pytest.mark.parametrize("name,defaults,kw", [
    ("svdq_gate_norm_modulate", NORM, PLACE),
    ("svdq_gate_norm_modulate", NORM, dict(PLACE, y=P(1))),             # the stream is its own block output
    ("svdq_gate_norm_modulate", NORM, dict(PLACE, gate=P(1), gr=4, gs=128)),   # and its own gate, row by row
    ("svdq_gate_norm_modulate", NORM, dict(PLACE, x=P(1), gate=P(1, 256), gr=4, gs=384, xs=384, hs=384)),  # between x's rows
    ("svdq_gate_norm_modulate", NORM, dict(PLACE, h=P(8), gate=P(1), gr=4, gs=128, scale=P(1), shift=P(1), mr=4, ms=128)),
    ("svdq_rope_axes", ROPE, dict(qo=P(1), qos=3072, ko=P(2), kos=3072))])
def test_places_that_are_allowed(name, defaults, kw):
    assert _call(name, defaults, kw) == NO_DEVICE


@pytest.mark.parametrize("kw", [
    dict(qo=P(1), qos=3072, k=P(1), ks=3072, kh=8), dict(q=P(2), qh=2, ko=P(2), kos=3072), dict(qo=P(1), qos=3072, ko=P(1, 1024), kos=3072),
    dict(q=P(1), k=P(1), qh=2, kh=2, qo=P(1), qos=3072, ko=P(1), kos=3072)])
def test_a_turn_in_place_shares_its_rows_with_nothing_else(kw):
    assert _call("svdq_rope_axes", ROPE, kw) == INVALID_VALUE


@pytest.mark.parametrize("kw", [dict(y=None), dict(y=None, h=None), dict(y=None, gate=None), dict(y=None, pw=None),
                                dict(x=None, y=None, h=None, z=None, zs=None)])
def test_no_rows_with_every_part(kw):
    """An empty batch has null rows, and its gate, weights and modulation as ever."""
    assert _call("svdq_gate_norm_modulate", NORM, dict(M=0, **kw)) == SUCCESS


@pytest.mark.parametrize("quantize", [None, "int8"])
def test_no_rows_through_the_binding(quantize):
    import torch
    import bit_diffusion_transformer_svdq_amd as pkg
    bf = torch.bfloat16
    x, v, w = torch.empty(0, 128, dtype=bf), torch.ones(2, 128, dtype=bf), torch.ones(128, dtype=bf)
    h, z = pkg.gate_norm_modulate(x, x, post_norm="rms", post_weight=w, gate=v, weight=w, scale=v, shift=v,
                                  quantize=quantize)
    assert h.shape == (0, 128) and (z if quantize is None else z[0]).shape == (0, 128)
    with pytest.raises(pkg.SvdqError):
        pkg.gate_norm_modulate(x, x, norm="none", scale=v)


@pytest.mark.parametrize("axes,status", [((-2,), INVALID_VALUE), ((), INVALID_VALUE), ((1 << 40,), NOT_SUPPORTED), ((1 << 62, 1 << 62), NOT_SUPPORTED),
                                         ((-2, 66), INVALID_VALUE), ((3,), INVALID_VALUE), ((258,), NOT_SUPPORTED), ((0,), INVALID_VALUE)])
def test_axes_are_refused_before_outputs_are_made(axes, status, monkeypatch):
    """Widths that the library refuses never decide how much memory is asked for, and
    widths past 64 bits do not wrap."""
    import torch
    import bit_diffusion_transformer_svdq_amd as pkg
    from bit_diffusion_transformer_svdq_amd import block
    asked = []
    real = torch.empty_strided
    monkeypatch.setattr(block.torch, "empty_strided", lambda shape, *a, **kw: (asked.append(shape), real(shape, *a, **kw))[1])
    with pytest.raises(pkg.SvdqError) as e:
        pkg.rope_axes_tables(torch.empty(0, len(axes)), axes)
    assert e.value.status == status
    assert all(len(s) == 2 and 0 <= s[1] <= 128 for s in asked)
    wide = tuple(axes) + ((1 << 64) + 64, 64 - (1 << 64))
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: pkg.rope_axes_tables(torch.empty(0, len(wide)), wide),
                 lambda: pkg.rope_axes(q, None, torch.empty(0, len(wide)), wide)):
        with pytest.raises(ValueError, match="axes"):
            call()


@pytest.mark.skipif(_gpu_visible(), reason="checks the no-GPU path")
@pytest.mark.parametrize("kw", [dict(xs=0, ys=0, hs=0), dict(xs=-8, ys=3, hs=1 << 60), dict(h=P(1), hs=0, xs=128), dict(h=P(1), hs=64, xs=7)])
def test_strides_of_one_row_are_not_read(kw):
    assert _call("svdq_gate_norm_modulate", NORM, dict(M=1, gr=1, gs=0, mr=1, ms=-5, **kw)) == NO_DEVICE


def test_one_row_over_another_is_still_refused():
    one = dict(M=1, gr=1, gs=0, mr=1, ms=0, xs=0, ys=0, hs=0)
    for kw in (dict(h=P(1, 16)), dict(h=P(2)), dict(h=P(6)), dict(z=P(1, 128)), dict(h=P(1), scale=P(1))):
        assert _call("svdq_gate_norm_modulate", NORM, dict(one, **kw)) == INVALID_VALUE
