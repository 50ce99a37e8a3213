"""The 8-bit linear (svdq_quantize_act_int8, svdq_w8a8_gemm) against the oracle.
Needs an MI355X.

Codes and scales are exact.  Y: the sum is exact; its fp32 value, the scale
product and the fma round by at most U each, the output by HALF_BF16; GELU adds
a few U of its argument (fp32 exponential and quotient: 8 fp32 ulp of |v|
covers them, since t exp(-t) <= 1/2)."""
import numpy as np
import pytest

import oracle as O
import oracle.block_oracle as B
from tests.block_util import HALF_BF16, U, bf16, check, dev, dev_bf16, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _acts(M, K, seed):
    g = np.random.default_rng([seed, M, K])
    x = g.standard_normal((M, K))
    x[:, g.permutation(K)[:max(1, K // 100)]] *= 30
    return bf16(x), g


def _smooth(g, K):
    return np.exp(0.7 * g.standard_normal(K)).astype(np.float32)


@pytest.mark.parametrize("M,K", [(1, 64), (3, 128), (5, 1088), (2, 4096), (9, 4160), (2, 8192), (3, 16384), (2, 16448),
                                 (1, 65536), (2100, 320), (2050, 3072), (2049, 4096), (300, 1920)])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantize_is_exact(M, K, smooth):
    import bit_diffusion_transformer_svdq_amd as P
    x, g = _acts(M, K, 1)
    sm = _smooth(g, K) if smooth else None
    q, s = P.quantize_act_int8(dev_bf16(x), None if sm is None else dev(sm))
    wq, ws = B.quantize_act_int8(x, sm)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


def test_quantize_reciprocals_are_correctly_rounded():
    """fl32(1/smooth) where a reciprocal is hardest to round: significands near all
    ones and all zeros, powers of two, the ends of the range."""
    import bit_diffusion_transformer_svdq_amd as P
    g = np.random.default_rng(5)
    bits = np.concatenate([
        (np.arange(1024, dtype=np.uint32) + np.uint32(0x3F800000)), np.uint32(0x3FFFFFFF) - np.arange(1024, dtype=np.uint32),
        g.integers(0x3F800000, 0x40000000, 8192 + 4096, dtype=np.uint32),
        (g.integers(20, 235, 1024, dtype=np.uint32) << np.uint32(23)) | np.uint32(0x7FFFFF),
        g.integers(0x08000000, 0x76000000, 1024, dtype=np.uint32)])
    K = bits.size
    assert K % 64 == 0
    sm = bits.view(np.float32)
    # one channel per row carries the row's value, so that its code is 127 and
    # its scale tells bf16(fl32(x mu)); rows of many such channels
    x = np.zeros((64, K))
    x[np.arange(K) % 64, np.arange(K)] = bf16(1 + g.random(K))
    wq, ws = B.quantize_act_int8(x, sm)
    q, s = P.quantize_act_int8(dev_bf16(x), dev(sm))
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quantize_odd_rows():
    """Zero rows, rows below the smallest scale, subnormal scales, ties, infinities
    and NaN: a bad row touches no other."""
    import bit_diffusion_transformer_svdq_amd as P
    K = 192
    x, _ = _acts(12, K, 2)
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2] *= 2.0 ** -122
    x[3, :] = np.arange(K) % 128 - 64 + 0.5   # exact halves after scaling by 127 / 127
    x[3, 0] = 127
    x[4, 7] = np.inf
    x[5, 9] = -np.inf
    x[6, 11] = np.nan
    x[7] *= 2.0 ** 120
    x = np.where(np.isfinite(x), bf16(np.where(np.isfinite(x), x, 0)), x)
    q, s = P.quantize_act_int8(dev_bf16(x))
    wq, ws = B.quantize_act_int8(np.asarray(dev_bf16(x).double().cpu()))
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True) and np.array_equal(q.cpu().numpy(), wq)
    w = np.ones((64, K), np.int8)
    y = host(P.w8a8_gemm(q, s, dev(w), dev(np.ones(64, np.float32))))
    assert np.isnan(y[4:7]).all() and np.isfinite(np.delete(y, (4, 5, 6), 0)).all()


def _gemm_case(M, N, K, seed, full=True):
    g = np.random.default_rng([seed, M, N, K])
    lo = -128 if full else -127
    qx, qw = g.integers(lo, 128, (M, K), dtype=np.int8), g.integers(lo, 128, (N, K), dtype=np.int8)
    sx = (np.exp(g.standard_normal(M)) * 1e-2).astype(np.float32)
    sw = (np.exp(g.standard_normal(N)) * 1e-3).astype(np.float32)
    return qx, sx, qw, sw, bf16(g.standard_normal(N))


def _check_gemm(y, qx, sx, qw, sw, b, epilogue):
    want, p = B.w8a8_gemm(qx, sx, qw, sw, b, epilogue)
    pre, _ = B.w8a8_gemm(qx, sx, qw, sw, b)
    err = 2 * U * np.abs(p) + U * np.abs(pre)
    if epilogue == "gelu_tanh":
        err = 1.2 * err + 16 * U * np.abs(pre)
    check(y, want, err)


@pytest.mark.parametrize("M,N,K", [
    (1, 64, 64), (1, 3072, 3072), (2, 192, 320), (16, 128, 1024), (17, 1088, 192), (33, 64, 65536), (64, 12288, 512),
    (64, 4160, 576), (48, 8256, 128), (31, 16448, 64),                                      # few tokens
    (65, 64, 64), (65, 128, 192), (127, 320, 640), (200, 448, 8192), (255, 3072, 3072), (257, 576, 448),
    (512, 1024, 1088), (1333, 2112, 1920), (700, 64, 16384), (2304, 9216, 320), (4100, 4160, 192)])
@pytest.mark.parametrize("epilogue", ["none", "gelu_tanh"])
def test_gemm(M, N, K, epilogue):
    import bit_diffusion_transformer_svdq_amd as P
    qx, sx, qw, sw, b = _gemm_case(M, N, K, 3)
    if epilogue == "gelu_tanh":
        sx *= np.float32(0.02)   # arguments of a few units, where GELU bends
    bias = b if (M + N) % 3 else None
    y = P.w8a8_gemm(dev(qx), dev(sx), dev(qw), dev(sw), dev_bf16(bias), epilogue=epilogue)
    _check_gemm(host(y), qx, sx, qw, sw, bias, epilogue)


@pytest.mark.parametrize("M", [2, 300])
def test_gelu_tails(M):
    """Arguments that are exact (small integers over 16), -7.9 to 7.9: the relative error
    is the function's own, (3.5 |t| + 7) 2^-24 with 2^t its exponential, and the
    rounding to bf16; fl32 constants and three roundings make up |t|'s share, the
    exponential, the reciprocal (an ulp each), a sum and a product the rest."""
    import bit_diffusion_transformer_svdq_amd as P
    qx, qw = np.zeros((M, 64), np.int8), np.zeros((256, 64), np.int8)
    qx[:, 5] = 1
    qw[:, 5] = np.arange(-128, 128)
    sx, sw = np.full(M, 2.0 ** -4, np.float32), np.ones(256, np.float32)
    y = host(P.w8a8_gemm(dev(qx), dev(sx), dev(qw), dev(sw), epilogue="gelu_tanh"))
    x = np.arange(-128, 128) / 16.0
    u = np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    want = x / (1 + np.exp(-2 * u))
    t = np.abs(2 * u * np.log2(np.e))
    assert (np.abs(y - want) <= (2.0 ** -8 / (1 + 2.0 ** -8) + 1.01 * (3.5 * t + 7) * U) * np.abs(want)).all()


@pytest.mark.parametrize("M", [3, 300])
def test_gemm_largest_sums(M):
    """Every product 2^14: the largest int32 sum, 2^30, stays exact."""
    import bit_diffusion_transformer_svdq_amd as P
    K = 65536
    qx, qw = np.full((M, K), -128, np.int8), np.full((64, K), -128, np.int8)
    y = host(P.w8a8_gemm(dev(qx), dev(np.ones(M, np.float32)), dev(qw), dev(np.ones(64, np.float32))))
    assert (y == 2.0 ** 30).all()


def test_gemm_repeats_bit_for_bit_and_leaves_the_workspace_clean():
    """K-splits through one workspace, other shapes in between; the arrival
    counters are back at zero."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd import _lib
    shapes = [(130, 256, 8192), (512, 3072, 3072), (70, 64, 16384)]
    needs = [_lib.lib().svdq_w8a8_gemm_workspace_size(*s) for s in shapes]
    assert any(needs)
    ws = torch.zeros(max(needs), dtype=torch.uint8, device="cuda")
    cases = [_gemm_case(*s, 4) for s in shapes]
    devs = [(dev(c[0]), dev(c[1]), dev(c[2]), dev(c[3])) for c in cases]
    first = [P.w8a8_gemm(*d, workspace=ws).clone() for d in devs]
    for _ in range(3):
        for d, f in zip(devs, first):
            assert torch.equal(P.w8a8_gemm(*d, workspace=ws), f)
    assert int(ws[:1 << 20].to(torch.int32).sum()) == 0
    for c, f in zip(cases, first):
        _check_gemm(host(f), *c[:4], None, "none")


def test_gemm_leaves_what_is_behind_its_rows():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    for M in (5, 130):
        qx, sx, qw, sw, b = _gemm_case(M, 192, 256, 6)
        buf = torch.full((M + 40, 192), 7.0, dtype=torch.bfloat16, device="cuda")
        P.w8a8_gemm(dev(qx), dev(sx), dev(qw), dev(sw), dev_bf16(b), out=buf[:M])
        assert bool((buf[M:] == 7).all())
        _check_gemm(host(buf[:M]), qx, sx, qw, sw, b, "none")


def test_codes_far_into_memory():
    """Rows whose codes lie beyond 4 GiB of the array's start."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    M, K, N = 70000, 65536, 64
    codes = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    qx, sx, qw, sw, _ = _gemm_case(100, N, K, 7)
    codes[-100:] = dev(qx)
    scales = torch.ones(M, device="cuda")
    scales[-100:] = dev(sx)
    y = P.w8a8_gemm(codes, scales, dev(qw), dev(sw))
    _check_gemm(host(y[-100:]), qx, sx, qw, sw, None, "none")
    assert not bool(y[:-100].any())


def test_packed_linear():
    """Packer, quantizer and product together, against the float product: the
    8-bit linear's own error is about one percent of it."""
    import bit_diffusion_transformer_svdq_amd as P
    M, K, N = 96, 512, 320
    x, g = _acts(M, K, 8)
    w = bf16(0.02 * g.standard_normal((N, K)))
    sm = np.sqrt(np.abs(x).max(0) / np.abs(w).max(0)).astype(np.float32)
    pk = P.pack_weights_int8(O.f64_to_bf16(w), sm)
    q, s = P.quantize_act_int8(dev_bf16(x), dev(sm))
    y = host(P.w8a8_gemm(q, s, dev(pk["w_codes"]), dev(pk["w_scales"])))
    wq, ws = B.quantize_act_int8(x, sm)
    _check_gemm(y, wq, ws, pk["w_codes"], pk["w_scales"], None, "none")
    ref = x @ w.T
    # both quantizers round by at most half a step per element
    step = 0.5 * (ws.astype(float)[:, None] * np.abs(pk["w_codes"].astype(float) * pk["w_scales"][:, None]).sum(1)[None]
                  + pk["w_scales"].astype(float)[None] * np.abs(x / sm).sum(1)[:, None]) + \
        0.25 * K * ws.astype(float)[:, None] * pk["w_scales"].astype(float)[None]
    xh = np.abs(x / sm) @ np.abs(w * sm).T
    assert (np.abs(y - ref) <= 1.02 * step + 2 * HALF_BF16 * xh).all()


@pytest.mark.parametrize("tile", [1, 114, 124, 222, 224, 323, 342, 432, 442])
@pytest.mark.parametrize("splits", [1, 2, 16])
def test_every_tile_and_split(tile, splits):
    """The same shapes on every kernel, tile and split give the same bits: one
    stage and less, an odd number of stages, a half one at the end, ragged
    tokens and channels."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    for M, N, K in [(9, 64, 64), (16, 192, 192), (70, 320, 448), (300, 576, 1088), (129, 448, 2176), (129, 448, 4096)]:
        if tile == 1 and M > 16:
            continue
        c = _gemm_case(M, N, K, 9)
        d = (dev(c[0]), dev(c[1]), dev(c[2]), dev(c[3]), dev_bf16(c[4]))
        want = P.w8a8_gemm(*d, epilogue="gelu_tanh")
        P.debug_set_w8a8_plan(tile, splits)
        try:
            got = P.w8a8_gemm(*d, epilogue="gelu_tanh")
        finally:
            P.debug_set_w8a8_plan()
        assert torch.equal(got, want), (M, N, K)
        _check_gemm(host(got), *c[:4], c[4], "gelu_tanh")
