"""C ABI checks of the block operators that need no GPU: refusals of svdq_quantize_act_int8,
svdq_w8a8_gemm, svdq_gate_norm_modulate, svdq_rope_axes_tables and svdq_rope_axes,
all reported before any HIP call, and the packer of the 8-bit linear."""
import ctypes

import numpy as np
import pytest

import oracle as O
from bit_diffusion_transformer_svdq_amd import _lib
from bit_diffusion_transformer_svdq_amd._lib import INVALID_VALUE, NO_DEVICE, NOT_SUPPORTED, SUCCESS, lib

NAN, INF = float("nan"), float("inf")


def P(i, off=0):
    """Fake device pointers, never dereferenced, 2^40 bytes apart."""
    return ctypes.c_void_p(((i + 1) << 40) + off)


def _gpu_visible():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


def _call(name, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    st = getattr(lib(), name)(*a.values())
    if st != SUCCESS:
        assert len(lib().svdq_last_error()) > 0
    return st


QUANT = dict(x=P(1), smooth=P(2), M=5, K=128, codes=P(3), scales=P(4), stream=None)
GEMM = dict(ac=P(1), asc=P(2), wc=P(3), wsc=P(4), bias=P(5), M=5, N=128, K=192, epilogue=1, y=P(6), ws=P(7),
            wsb=1 << 34, stream=None)
NORM = dict(x=P(1), stype=0, xs=128, y=P(2), ys=128, post=2, pw=P(3), gate=P(4), gr=2, gs=384, alpha=1.0, norm=1,
            w=P(5), scale=P(6), shift=P(7), mr=2, ms=384, eps=1e-6, M=4, C=128, h=P(8), hs=128, otype=1, smooth=P(9),
            z=P(10), zs=P(11), stream=None)
AXES = (ctypes.c_int64 * 3)(16, 56, 56)
TABLES = dict(pos=P(1), ptype=0, M=7, n=3, axes=AXES, theta=1e4, spectrum=0, cos=P(2), sin=P(3), stream=None)
ROPE = dict(q=P(1), qs=3072, qh=8, k=P(2), ks=3072, kh=2, D=128, M=6, pos=P(3), ptype=1, pr=3, n=3, axes=AXES, theta=1e4,
            spectrum=1, layout=1, qn=P(4), kn=P(5), eps=1e-6, qo=P(6), qos=1024, ko=P(7), kos=256, stream=None)


def _axes(*w):
    return dict(n=len(w), axes=(ctypes.c_int64 * max(1, len(w)))(*w))


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID_VALUE), (dict(codes=None), INVALID_VALUE), (dict(scales=None), INVALID_VALUE),
    (dict(x=P(1, 8)), INVALID_VALUE), (dict(smooth=P(2, 4)), INVALID_VALUE), (dict(M=-1), INVALID_VALUE),
    (dict(K=0), INVALID_VALUE), (dict(K=96), NOT_SUPPORTED), (dict(K=65600), NOT_SUPPORTED),
    (dict(M=(1 << 24) + 1), NOT_SUPPORTED), (dict(codes=P(1)), INVALID_VALUE), (dict(codes=P(1, 5 * 256 - 16)), INVALID_VALUE),
    (dict(scales=P(3, 16)), INVALID_VALUE), (dict(scales=P(2, 496)), INVALID_VALUE),
    (dict(M=0), SUCCESS), (dict(M=0, x=None, codes=None), SUCCESS), (dict(M=0, K=96), NOT_SUPPORTED)])
def test_quantize_refusals(kw, status):
    assert _call("svdq_quantize_act_int8", QUANT, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ac=None), INVALID_VALUE), (dict(asc=None), INVALID_VALUE), (dict(wc=None), INVALID_VALUE),
    (dict(wsc=None), INVALID_VALUE), (dict(y=None), INVALID_VALUE), (dict(N=96), NOT_SUPPORTED), (dict(K=100), NOT_SUPPORTED),
    (dict(N=0), INVALID_VALUE), (dict(K=65600), NOT_SUPPORTED), (dict(N=(1 << 20) + 64), NOT_SUPPORTED),
    (dict(epilogue=2), INVALID_VALUE), (dict(epilogue=-1), INVALID_VALUE), (dict(bias=P(5, 2)), INVALID_VALUE),
    (dict(wc=P(3, 8)), INVALID_VALUE), (dict(y=P(3, 128 * 192 - 16)), INVALID_VALUE), (dict(y=P(5)), INVALID_VALUE),
    (dict(M=0), SUCCESS), (dict(M=0, ac=None, y=None), SUCCESS), (dict(M=0, epilogue=7), INVALID_VALUE)])
def test_gemm_refusals(kw, status):
    assert _call("svdq_w8a8_gemm", GEMM, kw) == status


def test_gemm_workspace_rules():
    size = lib().svdq_w8a8_gemm_workspace_size
    assert size(4, 3072, 3072) == 0 and size(0, 64, 64) == 0 and size(5, 100, 64) == 0 and size(5, 64, 1 << 20) == 0
    big = dict(M=130, N=256, K=16384)
    need = size(130, 256, 16384)
    assert need > 1 << 20   # K is split over workgroups
    assert _call("svdq_w8a8_gemm", GEMM, dict(big, ws=None)) == INVALID_VALUE
    assert _call("svdq_w8a8_gemm", GEMM, dict(big, wsb=need - 1)) == INVALID_VALUE
    assert _call("svdq_w8a8_gemm", GEMM, dict(big, ws=P(7, 8))) == INVALID_VALUE
    assert _call("svdq_w8a8_gemm", GEMM, dict(big, ws=P(3), wsb=need)) == INVALID_VALUE
    assert _call("svdq_w8a8_gemm", GEMM, dict(big, ws=P(6), wsb=need)) == INVALID_VALUE
    hook = lib().svdq_debug_set_w8a8_plan
    for tile, splits in ((-1, 0), (2, 0), (43, 0), (999, 0), (0, -1), (0, 17)):
        assert hook(tile, splits) == INVALID_VALUE
    try:
        # 2 x 2 tiles of 128 x 128, four waves each, 4096 int32 per wave
        assert hook(224, 4) == SUCCESS and size(130, 256, 16384) == (1 << 20) + 4 * 4 * 4 * 4096 * 4
        assert hook(224, 1) == SUCCESS and size(130, 256, 16384) == 0
        assert hook(224, 16) == SUCCESS and size(130, 256, 256) == (1 << 20) + 4 * 4 * 2 * 4096 * 4   # two stages only
    finally:
        assert hook(0, 0) == SUCCESS


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID_VALUE), (dict(h=None), INVALID_VALUE), (dict(z=None), INVALID_VALUE), (dict(zs=None), INVALID_VALUE),
    (dict(C=100), NOT_SUPPORTED), (dict(C=72, xs=128), NOT_SUPPORTED), (dict(C=0), INVALID_VALUE), (dict(M=-1), INVALID_VALUE),
    (dict(C=32832, xs=32832, ys=32832, hs=32832, gs=32832, ms=32832), NOT_SUPPORTED), (dict(M=(1 << 24) + 2), NOT_SUPPORTED),
    (dict(stype=2), INVALID_VALUE), (dict(post=3), INVALID_VALUE), (dict(norm=-1), INVALID_VALUE), (dict(otype=2), INVALID_VALUE),
    (dict(eps=-1e-6), INVALID_VALUE), (dict(eps=NAN), INVALID_VALUE), (dict(eps=INF), INVALID_VALUE),
    (dict(alpha=NAN), INVALID_VALUE), (dict(alpha=INF), INVALID_VALUE),
    (dict(xs=120), INVALID_VALUE), (dict(xs=132), NOT_SUPPORTED), (dict(ys=0), INVALID_VALUE), (dict(gs=64), INVALID_VALUE),
    (dict(ms=129), NOT_SUPPORTED), (dict(hs=129), NOT_SUPPORTED), (dict(xs=1 << 41), NOT_SUPPORTED),
    (dict(gr=3), INVALID_VALUE), (dict(gr=0), INVALID_VALUE), (dict(mr=8), INVALID_VALUE), (dict(gr=8), INVALID_VALUE),
    (dict(y=None), INVALID_VALUE),                                              # a gate without a block output
    (dict(y=None, gate=None, pw=None), INVALID_VALUE),                          # a post norm without one
    (dict(y=None, gate=None, pw=None, post=0, norm=0, w=None, scale=None, shift=None, smooth=None, otype=0), INVALID_VALUE),
    (dict(post=0), INVALID_VALUE),                                              # post_weight without its norm
    (dict(norm=0), INVALID_VALUE), (dict(norm=0, w=None), INVALID_VALUE),
    (dict(norm=0, w=None, scale=None, shift=None, smooth=None), INVALID_VALUE),  # 8-bit output without a norm
    (dict(otype=0), INVALID_VALUE),                                             # smooth without 8-bit output
    (dict(x=P(1, 8)), INVALID_VALUE), (dict(gate=P(4, 2)), INVALID_VALUE), (dict(zs=P(11, 4)), INVALID_VALUE),
    (dict(z=P(1)), INVALID_VALUE), (dict(h=P(2)), INVALID_VALUE), (dict(h=P(1, 16)), INVALID_VALUE),
    (dict(h=P(1), hs=256), INVALID_VALUE),                                      # x's address, another stride
    (dict(h=P(4, 256)), INVALID_VALUE), (dict(z=P(8)), INVALID_VALUE), (dict(zs=P(10, 16)), INVALID_VALUE),
    (dict(stype=1, xs=128, x=P(1), y=P(1), ys=256, h=P(1), hs=128), INVALID_VALUE),
    (dict(M=0), SUCCESS), (dict(M=0, x=None, y=None, gate=None, pw=None, h=None, z=None, zs=None), SUCCESS),
    (dict(M=0, norm=5), INVALID_VALUE)])
def test_norm_refusals(kw, status):
    assert _call("svdq_gate_norm_modulate", NORM, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(pos=None), INVALID_VALUE), (dict(cos=None), INVALID_VALUE), (dict(sin=None), INVALID_VALUE), (dict(ptype=2), INVALID_VALUE),
    (dict(M=-1), INVALID_VALUE), (dict(theta=1.0), INVALID_VALUE), (dict(theta=NAN), INVALID_VALUE), (dict(theta=INF), INVALID_VALUE),
    (dict(spectrum=2), INVALID_VALUE), (dict(n=0), INVALID_VALUE), (dict(axes=None), INVALID_VALUE), (_axes(16, 0), INVALID_VALUE),
    (_axes(16, 3), INVALID_VALUE), (_axes(-2), INVALID_VALUE), (_axes(*[2] * 9), NOT_SUPPORTED), (_axes(200, 64), NOT_SUPPORTED),
    (_axes(1 << 40), NOT_SUPPORTED), (dict(cos=P(3, 16)), INVALID_VALUE), (dict(sin=P(1)), INVALID_VALUE),
    (dict(pos=P(1, 4)), INVALID_VALUE), (dict(M=(1 << 24) + 1), NOT_SUPPORTED), (dict(M=0), SUCCESS), (dict(M=0, pos=None), SUCCESS)])
def test_table_refusals(kw, status):
    assert _call("svdq_rope_axes_tables", TABLES, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID_VALUE), (dict(k=None), INVALID_VALUE), (dict(pos=None), INVALID_VALUE), (dict(qo=None), INVALID_VALUE),
    (dict(ko=None), INVALID_VALUE), (dict(qh=0), INVALID_VALUE), (dict(kh=-1), INVALID_VALUE), (dict(D=100), NOT_SUPPORTED),
    (dict(D=264), NOT_SUPPORTED), (dict(qh=4097), NOT_SUPPORTED), (dict(layout=2), INVALID_VALUE), (dict(ptype=-1), INVALID_VALUE),
    (dict(D=120), INVALID_VALUE),                                               # 128 channels of axes
    (_axes(16, 54, 56), NOT_SUPPORTED),                                         # halves of 63 channels
    (dict(eps=-1.0), INVALID_VALUE), (dict(kn=None), INVALID_VALUE), (dict(qn=None), INVALID_VALUE), (dict(kh=0), INVALID_VALUE),
    (dict(pr=0), INVALID_VALUE), (dict(pr=4), INVALID_VALUE), (dict(pr=12), INVALID_VALUE), (dict(qs=1016), INVALID_VALUE),
    (dict(qs=3076), NOT_SUPPORTED), (dict(kos=255), INVALID_VALUE), (dict(qos=1 << 39), NOT_SUPPORTED),
    (dict(q=P(1, 8)), INVALID_VALUE), (dict(qn=P(4, 8)), INVALID_VALUE),
    (dict(qo=P(1)), INVALID_VALUE),                                             # q's address, another stride
    (dict(qo=P(1, 16), qos=3072), INVALID_VALUE), (dict(qo=P(2), qos=3072), INVALID_VALUE), (dict(ko=P(1), kos=3072), INVALID_VALUE),
    (dict(qo=P(7)), INVALID_VALUE), (dict(qo=P(3)), INVALID_VALUE), (dict(ko=P(4)), INVALID_VALUE),
    (dict(q=P(1), k=P(1, 2032), qo=P(1), qos=3072, ko=P(1, 2032), kos=3072), INVALID_VALUE),   # q's last channels are k's first
    (dict(M=0), SUCCESS), (dict(M=0, q=None, k=None, qo=None, ko=None, pos=None), SUCCESS), (dict(M=0, layout=9), INVALID_VALUE)])
def test_rope_refusals(kw, status):
    assert _call("svdq_rope_axes", ROPE, kw) == status


@pytest.mark.skipif(_gpu_visible(), reason="checks the no-GPU path")
def test_good_calls_reach_the_device_check():
    good = [("svdq_quantize_act_int8", QUANT, {}), ("svdq_quantize_act_int8", QUANT, dict(smooth=None, M=1 << 24, K=64)),
            ("svdq_w8a8_gemm", GEMM, {}), ("svdq_w8a8_gemm", GEMM, dict(bias=None, ws=None, wsb=0, M=3, epilogue=0)),
            ("svdq_gate_norm_modulate", NORM, {}),
            ("svdq_gate_norm_modulate", NORM, dict(h=P(1))),                    # the stream in place
            ("svdq_gate_norm_modulate", NORM, dict(gr=1, gs=0, mr=4, alpha=0.0, eps=0.0)),
            # chunks of one modulation buffer, h a column block beside y
            ("svdq_gate_norm_modulate", NORM, dict(gate=P(4), scale=P(4, 256), shift=P(4, 512), y=P(2), ys=256, h=P(2, 256), hs=256)),
            ("svdq_gate_norm_modulate", NORM, dict(y=None, gate=None, pw=None, post=0, h=None)),
            ("svdq_gate_norm_modulate", NORM, dict(norm=0, w=None, scale=None, shift=None, smooth=None, otype=0, z=None, zs=None)),
            ("svdq_rope_axes_tables", TABLES, {}), ("svdq_rope_axes_tables", TABLES, _axes(*[32] * 8)),
            ("svdq_rope_axes", ROPE, {}), ("svdq_rope_axes", ROPE, dict(k=None, kh=0, ko=None, kn=None)),
            # Q and K of one buffer turned in place
            ("svdq_rope_axes", ROPE, dict(q=P(1), k=P(1, 2048), qo=P(1), qos=3072, ko=P(1, 2048), kos=3072))]
    for name, defaults, kw in good:
        assert _call(name, defaults, kw) == NO_DEVICE, (name, kw)


@pytest.mark.parametrize("N,K,smooth", [(1, 1, False), (3, 7, True), (70, 129, True), (64, 192, False)])
def test_packer(N, K, smooth):
    """Codes and scales by the definition in double, a zero row, ties to even."""
    import bit_diffusion_transformer_svdq_amd as pkg
    g = np.random.default_rng([N, K])
    bits = O.f64_to_bf16(0.02 * g.standard_normal((N, K)))
    if N > 2:
        bits[1] = 0
    if N > 60:
        bits[2] = O.f64_to_bf16((np.arange(K) % 128 - 64 + 0.5) / 4)
        bits[2, 0] = O.f64_to_bf16(np.array([127 / 4]))[0]
    lam = np.exp(g.standard_normal(K)).astype(np.float32) if smooth else None
    pk = pkg.pack_weights_int8(bits, lam)
    w = O.bf16_to_f64(bits) * (1.0 if lam is None else lam.astype(np.float64))
    s = (np.abs(w).max(1) / 127).astype(np.float32)
    q = np.where(s[:, None] > 0, np.rint(w / np.where(s > 0, s, 1).astype(np.float64)[:, None]), 0)
    assert np.array_equal(pk["w_scales"], s) and np.array_equal(pk["w_codes"], q.astype(np.int8))
    assert np.abs(pk["w_codes"]).max() <= 127


def test_packer_refusals(monkeypatch):
    import bit_diffusion_transformer_svdq_amd as pkg
    w = np.zeros((4, 8), np.uint16)
    with pytest.raises(ValueError):
        pkg.pack_weights_int8(w, np.ones(7, np.float32))
    for bad in (0x7F80, 0x7FC0):
        x = w.copy()
        x[3, 5] = bad
        with pytest.raises(pkg.SvdqError):
            pkg.pack_weights_int8(x)
    with pytest.raises(pkg.SvdqError):
        pkg.pack_weights_int8(np.full((2, 8), 0x3F80, np.uint16), np.full(8, np.inf, np.float32))
    with pytest.raises(pkg.SvdqError):
        pkg.pack_weights_int8(np.zeros((0, 8), np.uint16))
    monkeypatch.setenv("SVDQ_PACK_THREADS", "1")
    g = np.random.default_rng(1)
    x = O.f64_to_bf16(g.standard_normal((40, 24)))
    one = pkg.pack_weights_int8(x)
    monkeypatch.setenv("SVDQ_PACK_THREADS", "7")
    many = pkg.pack_weights_int8(x)
    assert np.array_equal(one["w_codes"], many["w_codes"]) and np.array_equal(one["w_scales"], many["w_scales"])


def test_binding_names_the_block_operators():
    import bit_diffusion_transformer_svdq_amd as pkg
    for n in ("quantize_act_int8", "w8a8_gemm", "pack_weights_int8", "gate_norm_modulate", "rope_axes", "rope_axes_tables"):
        assert n in pkg.__all__ and callable(getattr(pkg, n))
        assert "svdq_" + n.replace("pack_weights_int8", "pack_weights_int8") in _lib.SIGNATURES
    with pytest.raises(AttributeError):
        pkg.no_such_operator


def test_host_tensors_are_refused():
    import torch
    import bit_diffusion_transformer_svdq_amd as pkg
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 64, dtype=torch.int8)
    s = torch.zeros(2)
    for call in (lambda: pkg.quantize_act_int8(x), lambda: pkg.w8a8_gemm(c, s, c, s), lambda: pkg.gate_norm_modulate(x),
                 lambda: pkg.rope_axes(x.view(2, 1, 64), None, torch.zeros(2, 1), (64,)),
                 lambda: pkg.rope_axes_tables(torch.zeros(2, 1), (64,))):
        with pytest.raises(ValueError, match="device tensor"):
            call()
