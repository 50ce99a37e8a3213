"""C ABI checks of the 8-bit floating-point linear and the gated product that need no GPU:
refusals, all reported before any HIP call, workspace rules, the packer, and the
binding's names."""
import ctypes

import numpy as np
import pytest

import oracle as O
import oracle.fp8_oracle as F
from bit_diffusion_transformer_svdq_amd import _lib
from bit_diffusion_transformer_svdq_amd._lib import INVALID_VALUE, NO_DEVICE, NOT_SUPPORTED, SUCCESS, lib
from tests.test_block_abi_host import NORM, P, _call, _gpu_visible

QUANT = dict(x=P(1), smooth=P(2), M=5, K=320, codes=P(3), scales=P(4), ss=5, stream=None)
GEMM = dict(ac=P(1), asc=P(2), ss=5, wc=P(3), wsc=P(4), bias=P(5), M=5, N=128, K=320, epilogue=1, y=P(6), ws=P(7),
            wsb=1 << 34, stream=None)
GATED = dict(ac=P(1), asc=P(2), ss=5, gc=P(3), gs=P(4), uc=P(5), us=P(6), gb=P(7), ub=P(8), M=5, F=192, K=320, act=0, otype=1,
             smooth=P(9), out=P(10), os=P(11), oss=5, ws=P(12), wsb=1 << 34, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID_VALUE), (dict(codes=None), INVALID_VALUE), (dict(scales=None), INVALID_VALUE),
    (dict(x=P(1, 8)), INVALID_VALUE), (dict(smooth=P(2, 4)), INVALID_VALUE), (dict(scales=P(4, 2)), INVALID_VALUE),
    (dict(M=-1), INVALID_VALUE), (dict(K=0), INVALID_VALUE), (dict(K=96), NOT_SUPPORTED), (dict(K=65600), NOT_SUPPORTED),
    (dict(M=(1 << 24) + 1), NOT_SUPPORTED), (dict(ss=4), INVALID_VALUE), (dict(ss=-8), INVALID_VALUE),
    (dict(ss=(1 << 37) + 1), NOT_SUPPORTED),
    (dict(codes=P(1)), INVALID_VALUE), (dict(codes=P(1, 5 * 640 - 16)), INVALID_VALUE), (dict(codes=P(2)), INVALID_VALUE),
    (dict(scales=P(3, 16)), INVALID_VALUE), (dict(scales=P(2, 1264)), INVALID_VALUE),
    (dict(ss=1000, scales=P(3, -8000)), INVALID_VALUE),                      # the third row of scales in the codes
    (dict(M=0), SUCCESS), (dict(M=0, x=None, codes=None, scales=None, ss=-1), SUCCESS), (dict(M=0, K=96), NOT_SUPPORTED)])
def test_quantize_refusals(kw, status):
    assert _call("svdq_quantize_act_fp8", QUANT, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ac=None), INVALID_VALUE), (dict(asc=None), INVALID_VALUE), (dict(wc=None), INVALID_VALUE),
    (dict(wsc=None), INVALID_VALUE), (dict(y=None), INVALID_VALUE), (dict(N=96), NOT_SUPPORTED), (dict(K=100), NOT_SUPPORTED),
    (dict(N=0), INVALID_VALUE), (dict(K=65600), NOT_SUPPORTED), (dict(N=(1 << 20) + 64), NOT_SUPPORTED), (dict(M=-5), INVALID_VALUE),
    (dict(ss=4), INVALID_VALUE), (dict(ss=1 << 38), NOT_SUPPORTED),
    (dict(epilogue=2), INVALID_VALUE), (dict(epilogue=-1), INVALID_VALUE), (dict(bias=P(5, 2)), INVALID_VALUE),
    (dict(wc=P(3, 8)), INVALID_VALUE), (dict(wsc=P(4, 4)), INVALID_VALUE), (dict(y=P(3, 128 * 320 - 16)), INVALID_VALUE),
    (dict(y=P(5)), INVALID_VALUE), (dict(y=P(2, 32)), INVALID_VALUE), (dict(y=P(4)), INVALID_VALUE), (dict(y=P(1)), INVALID_VALUE),
    (dict(M=0), SUCCESS), (dict(M=0, ac=None, y=None, ss=0), SUCCESS), (dict(M=0, epilogue=7), INVALID_VALUE)])
def test_gemm_refusals(kw, status):
    assert _call("svdq_fp8_gemm", GEMM, kw) == status


@pytest.mark.parametrize("kw,status", [
    *[(dict([(n, None)]), INVALID_VALUE) for n in ("ac", "asc", "gc", "gs", "uc", "us", "out", "os")],
    *[(dict([(n, P(i, 2 if n in ("asc", "os") else 8))]), INVALID_VALUE)
      for i, n in enumerate(("ac", "asc", "gc", "gs", "uc", "us", "gb", "ub", "smooth", "out", "os"), 1)],
    (dict(F=96), NOT_SUPPORTED), (dict(K=100), NOT_SUPPORTED), (dict(F=-64), INVALID_VALUE), (dict(F=(1 << 20) + 64), NOT_SUPPORTED),
    (dict(act=2), INVALID_VALUE), (dict(act=-1), INVALID_VALUE), (dict(otype=2), INVALID_VALUE), (dict(otype=0), INVALID_VALUE),
    (dict(ss=0), INVALID_VALUE), (dict(oss=4), INVALID_VALUE), (dict(oss=1 << 38), NOT_SUPPORTED),
    *[(dict(out=P(i)), INVALID_VALUE) for i in range(1, 10)], *[(dict(os=P(i)), INVALID_VALUE) for i in range(1, 11)],
    (dict(os=P(10, 5 * 192 - 16)), INVALID_VALUE), (dict(out=P(11)), INVALID_VALUE),
    (dict(M=0), SUCCESS), (dict(M=0, ac=None, out=None, os=None), SUCCESS), (dict(M=0, act=7), INVALID_VALUE),
    (dict(M=0, otype=0), INVALID_VALUE)])
def test_gated_refusals(kw, status):
    assert _call("svdq_fp8_gated_gemm", GATED, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(C=72, xs=128), NOT_SUPPORTED), (dict(zs=None), INVALID_VALUE), (dict(z=P(1)), INVALID_VALUE), (dict(zs=P(10, 16)), INVALID_VALUE),
    (dict(zs=P(2, 1008)), INVALID_VALUE), (dict(otype=4), INVALID_VALUE), (dict(norm=0, w=None, scale=None, shift=None, smooth=None), INVALID_VALUE),
    (dict(M=0), SUCCESS)])
def test_norm_into_codes_refusals(kw, status):
    assert _call("svdq_gate_norm_modulate", NORM, dict(dict(otype=3), **kw)) == status
    # the scales of 3 blocks: 4 tokens each
    wide = dict(otype=3, C=320, xs=320, ys=320, hs=320, gs=320, ms=320)
    assert _call("svdq_gate_norm_modulate", NORM, dict(wide, zs=P(9, 1280 - 48))) == INVALID_VALUE
    assert _call("svdq_gate_norm_modulate", NORM, dict(wide, zs=P(9, -32))) == INVALID_VALUE


def test_workspace_rules():
    size, gated = lib().svdq_fp8_gemm_workspace_size, lib().svdq_fp8_gated_gemm_workspace_size
    assert size(4, 1536, 1536) == 0 and size(0, 64, 64) == 0 and size(5, 100, 64) == 0 and size(5, 64, 1 << 20) == 0
    assert gated(4, 1536, 1536, 0) == 0 and gated(0, 64, 64, 1) == 0 and gated(4, 64, 64, 2) == 0
    # few tokens into codes: a counter per block of features, fp32 rows of 16 tokens
    assert gated(4, 320, 1536, 1) == (1 << 20) + 320 * 16 * 4
    big = dict(M=130, N=256, K=16384, ss=130)
    need = size(130, 256, 16384)
    assert need > 1 << 20   # K is split over workgroups
    assert _call("svdq_fp8_gemm", GEMM, dict(big, ws=None)) == INVALID_VALUE
    assert _call("svdq_fp8_gemm", GEMM, dict(big, wsb=need - 1)) == INVALID_VALUE
    assert _call("svdq_fp8_gemm", GEMM, dict(big, ws=P(7, 8))) == INVALID_VALUE
    for p in (1, 2, 3, 4, 5, 6):
        assert _call("svdq_fp8_gemm", GEMM, dict(big, ws=P(p), wsb=need)) == INVALID_VALUE
    for p in range(1, 12):
        assert _call("svdq_fp8_gated_gemm", GATED, dict(ws=P(p))) == INVALID_VALUE
    assert _call("svdq_fp8_gated_gemm", GATED, dict(ws=None)) == INVALID_VALUE
    assert _call("svdq_fp8_gated_gemm", GATED, dict(wsb=(1 << 20) + 192 * 64 - 1)) == INVALID_VALUE
    hook = lib().svdq_debug_set_fp8_plan
    for tile, splits in ((-1, 0), (2, 0), (43, 0), (999, 0), (0, -1), (0, 17)):
        assert hook(tile, splits) == INVALID_VALUE
    try:
        # 2 x 2 tiles of 128 x 128, 16384 fp32 per tile and split
        assert hook(224, 4) == SUCCESS and size(130, 256, 16384) == (1 << 20) + 4 * 4 * 16384 * 4
        assert hook(224, 1) == SUCCESS and size(130, 256, 16384) == 0
        assert hook(224, 16) == SUCCESS and size(130, 256, 256) == (1 << 20) + 4 * 2 * 16384 * 4   # two blocks only
        assert gated(130, 128, 16384, 0) == (1 << 20) + 2 * 2 * 16 * 16384 * 4   # 64 features a tile
    finally:
        assert hook(0, 0) == SUCCESS


@pytest.mark.skipif(_gpu_visible(), reason="checks the no-GPU path")
def test_good_calls_reach_the_device_check():
    good = [("svdq_quantize_act_fp8", QUANT, {}), ("svdq_quantize_act_fp8", QUANT, dict(smooth=None, M=1 << 24, K=64, ss=-3)),
            ("svdq_quantize_act_fp8", QUANT, dict(ss=1000, scales=P(4, 4))),     # from the second token on
            ("svdq_fp8_gemm", GEMM, dict(ss=1000, asc=P(2, 12))), ("svdq_fp8_gated_gemm", GATED, dict(ss=100, asc=P(2, 4), oss=100, os=P(11, 8))),
            ("svdq_fp8_gemm", GEMM, {}), ("svdq_fp8_gemm", GEMM, dict(bias=None, ws=None, wsb=0, M=3, epilogue=0)),
            ("svdq_fp8_gemm", GEMM, dict(K=64, ss=0)),                           # one row of scales has no stride
            ("svdq_fp8_gated_gemm", GATED, {}), ("svdq_fp8_gated_gemm", GATED, dict(otype=0, smooth=None, os=None, oss=0, ws=None, wsb=0)),
            # the scales written beside those read, rows of one larger array
            ("svdq_fp8_gated_gemm", GATED, dict(ss=64, asc=P(2), os=P(2, 128), oss=64)),
            ("svdq_gate_norm_modulate", NORM, dict(otype=3)), ("svdq_gate_norm_modulate", NORM, dict(otype=3, h=P(1)))]
    for name, defaults, kw in good:
        assert _call(name, defaults, kw) == NO_DEVICE, (name, kw)


@pytest.mark.parametrize("N,K,smooth", [(1, 1, False), (3, 7, True), (130, 129, True), (64, 192, False), (257, 300, True)])
def test_packer(N, K, smooth):
    """Codes and scales by the definition in double, a zero block, ties to the even code,
    values below the least."""
    import bit_diffusion_transformer_svdq_amd as pkg
    g = np.random.default_rng([N, K])
    w = 0.02 * g.standard_normal((N, K))
    if N > 128:
        w[128:] = 0
    if K > 130:
        w[:, 130:] *= np.exp(-8 * g.random((N, K - 130)))
    if K == 192:
        mids = (F.VALUES[:127][:-1] + F.VALUES[:127][1:]) / 2
        w[:, :126], w[:, 126], w[:, 127] = mids, 448, 0.0
    bits = O.f64_to_bf16(w)
    lam = np.exp(g.standard_normal(K)).astype(np.float32) if smooth else None
    pk = pkg.pack_weights_fp8(bits, lam)
    codes, scales = F.pack_weights_fp8(O.bf16_to_f64(bits), lam)
    assert np.array_equal(pk["w_scales"], scales) and np.array_equal(pk["w_codes"], codes)


def test_packer_refusals(monkeypatch):
    import bit_diffusion_transformer_svdq_amd as pkg
    w = np.zeros((4, 8), np.uint16)
    with pytest.raises(ValueError):
        pkg.pack_weights_fp8(w, np.ones(7, np.float32))
    for bad in (0x7F80, 0x7FC0):
        x = w.copy()
        x[3, 5] = bad
        with pytest.raises(pkg.SvdqError):
            pkg.pack_weights_fp8(x)
    with pytest.raises(pkg.SvdqError):
        pkg.pack_weights_fp8(np.full((2, 8), 0x3F80, np.uint16), np.full(8, np.inf, np.float32))
    with pytest.raises(pkg.SvdqError):
        pkg.pack_weights_fp8(np.zeros((0, 8), np.uint16))
    g = np.random.default_rng(1)
    x = O.f64_to_bf16(g.standard_normal((700, 24)))
    monkeypatch.setenv("SVDQ_PACK_THREADS", "1")
    one = pkg.pack_weights_fp8(x)
    monkeypatch.setenv("SVDQ_PACK_THREADS", "7")
    many = pkg.pack_weights_fp8(x)
    assert np.array_equal(one["w_codes"], many["w_codes"]) and np.array_equal(one["w_scales"], many["w_scales"])


def test_binding_names_the_operators():
    import bit_diffusion_transformer_svdq_amd as pkg
    for n in ("quantize_act_fp8", "fp8_gemm", "fp8_gated_gemm", "gated_ffn_fp8", "pack_weights_fp8", "debug_set_fp8_plan"):
        assert n in pkg.__all__ and callable(getattr(pkg, n))
    for n in ("quantize_act_fp8", "fp8_gemm", "fp8_gated_gemm", "pack_weights_fp8"):
        assert "svdq_" + n in _lib.SIGNATURES


def test_host_tensors_and_no_rows():
    import torch
    import bit_diffusion_transformer_svdq_amd as pkg
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    x = torch.zeros(2, 64, dtype=bf)
    c, s = torch.zeros(2, 64).to(f8), torch.zeros(1, 2)
    w, z = torch.zeros(64, 64).to(f8), torch.zeros(1, 1)
    for call in (lambda: pkg.quantize_act_fp8(x), lambda: pkg.fp8_gemm(c, s, w, z), lambda: pkg.fp8_gated_gemm(c, s, w, z, w, z),
                 lambda: pkg.gate_norm_modulate(x, quantize="fp8")):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    # an empty batch needs no device
    q, s = pkg.quantize_act_fp8(x[:0])
    assert q.shape == (0, 64) and s.shape == (1, 0) and q.dtype is f8
    h, (q, s) = pkg.gate_norm_modulate(x[:0], quantize="fp8")
    assert h is None and q.shape == (0, 64) and s.shape == (1, 0)


@pytest.mark.parametrize("v", [0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 448.0, 463.9, -5 * 2.0 ** -10, 0.9375, 0.96875])
def test_oracle_codes(v):
    """The oracle's codes against torch's own conversion."""
    import torch
    t = torch.tensor([v, -v]).to(torch.float8_e4m3fn)
    assert np.array_equal(F.encode(np.array([v, -v])), t.view(torch.uint8).numpy())
    assert np.array_equal(F.decode(F.encode(np.array([v, -v]))), t.double().numpy())


def test_oracle_codes_of_random_values():
    import torch
    g = np.random.default_rng(0)
    v = (g.standard_normal(20000) * np.exp(g.uniform(-8, 4.5, 20000))).astype(np.float32)
    v = v[np.abs(v) < 448]
    assert np.array_equal(F.encode(v), torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    every = np.arange(256, dtype=np.uint8)
    assert np.array_equal(F.decode(every), torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_oracle_is_the_float_product_for_whole_numbers():
    """Whole numbers that e4m3 holds, one of 448 in each block so that scales are exact
    enough to be 1: the oracle's product is the integers' own, and a gate of zeros gives
    zeros."""
    g = np.random.default_rng(2)
    x, w = g.integers(-4, 5, (5, 320)).astype(float), g.integers(-4, 5, (192, 320)).astype(float)
    x[:, ::128], w[::64, ::64] = 448, 448
    xq, wq = F.quantize(x), F.pack_weights_fp8(w)
    assert (xq[1] == 1).all() and (wq[1] == 1).all()
    assert np.array_equal(F.fp8_gemm(*xq, *wq), x @ w.T)
    assert not F.fp8_gated_gemm(*xq, (np.zeros((192, 320), np.uint8), wq[1]), wq).any()
