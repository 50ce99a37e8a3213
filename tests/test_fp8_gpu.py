"""The 8-bit floating-point linear (svdq_quantize_act_fp8, svdq_fp8_gemm) against the
oracle.  Needs an MI355X.  Codes and scales are exact; bounds of the products:
tests/fp8_util.py."""
import numpy as np
import pytest

import oracle as O
import oracle.fp8_oracle as F
from tests.block_util import HALF_BF16, U, bf16, check, dev, dev_bf16, host
from tests.fp8_util import act_bound, acts, cut_bound, dev_codes, host_codes, product_bound, tokens, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _same(got, want):
    assert np.array_equal(got[1].cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(host_codes(got[0]), want[0])


@pytest.mark.parametrize("M,K", [(1, 64), (3, 128), (5, 1088), (17, 192), (2, 4096), (9, 4160), (33, 512), (2, 65536), (4133, 576),
                                 (20000, 64), (300, 1920)])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantize_is_exact(M, K, smooth):
    import bit_diffusion_transformer_svdq_amd as P
    x, g = acts(M, K, 1)
    sm = np.exp(0.7 * g.standard_normal(K)).astype(np.float32) if smooth else None
    _same(P.quantize_act_fp8(dev_bf16(x), None if sm is None else dev(sm)), F.quantize_act_fp8(x, sm))


def test_quantize_every_border():
    """Values on and next to the borders between neighbouring codes, subnormal ones among
    them: a block's largest value is 448, so that its scale is fl32(448 fl32(1/448)) = 1."""
    import bit_diffusion_transformer_svdq_amd as P
    top = F.VALUES[:127]
    mids = (top[:-1] + top[1:]) / 2
    v = np.concatenate([top, mids, bf16(mids * (1 + 2.0 ** -8)), bf16(mids * (1 - 2.0 ** -8))])
    v = bf16(np.concatenate([v, -v, [2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -10, -0.0]]))
    rows = np.zeros((-(-v.size // 120), 128))
    for i in range(rows.shape[0]):
        part = v[120 * i:120 * (i + 1)]
        rows[i, :part.size] = part
        rows[i, 127] = 448
    want = F.quantize_act_fp8(rows)
    assert (want[1] == 1).all()
    _same(P.quantize_act_fp8(dev_bf16(rows)), want)


def test_quantize_odd_rows():
    """Zero blocks, blocks below the smallest scale, subnormal scales, infinities and NaN:
    a bad block touches no other, and its token's row of Y alone is NaN."""
    import bit_diffusion_transformer_svdq_amd as P
    K = 320
    x, _ = acts(12, K, 2)
    x[0] = 0
    x[1, :128] = 0
    x[2] *= 2.0 ** -130
    x[3] *= 2.0 ** -122
    x[4, 7], x[5, 200], x[6, 319] = np.inf, -np.inf, np.nan
    x[7] *= 2.0 ** 120
    x[8, 256:] *= 2.0 ** -126
    x = np.where(np.isfinite(x), bf16(np.where(np.isfinite(x), x, 0)), x)
    q, s = P.quantize_act_fp8(dev_bf16(x))
    _same((q, s), F.quantize_act_fp8(np.asarray(dev_bf16(x).double().cpu())))
    w = np.full((64, K), 0x38, np.uint8)  # ones
    for M in (12, 7):
        y = host(P.fp8_gemm(q[:M], s[:, :M], dev_codes(w), dev(np.ones((1, 3), np.float32))))
        assert np.isnan(y[4:7]).all() and np.isfinite(np.delete(y, (4, 5, 6), 0)).all()
    big = dev_bf16(np.repeat(x, 10, 0))
    q, s = P.quantize_act_fp8(big)
    y = host(P.fp8_gemm(q, s, dev_codes(w), dev(np.ones((1, 3), np.float32))))
    bad = np.repeat(np.isin(np.arange(12), (4, 5, 6)), 10)
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


def _check_gemm(y, x, w, b, epilogue, cut=False):
    K = x[0].shape[1]
    v, mags = F.product(*x, *w, b)
    err = product_bound(K, mags, v) + (cut_bound(*x, *w) if cut else 0)
    if epilogue == "gelu_tanh":
        err, v = act_bound(v, err), F.gelu_tanh(v)
    check(y, v, err)


def _dev(x, w):
    return dev_codes(x[0]), dev(x[1]), dev_codes(w[0]), dev(w[1])


SHAPES = [(1, 64, 64), (1, 1536, 1536), (2, 192, 320), (16, 128, 1024), (16, 4160, 192), (7, 64, 65536), (5, 8256, 128), (3, 16448, 64),
          (17, 1088, 192), (33, 64, 65536), (64, 12288, 512), (64, 4160, 576), (65, 64, 64), (65, 128, 192), (127, 320, 640),
          (200, 448, 8192), (255, 1536, 1536), (257, 576, 448), (512, 1024, 1088), (1333, 2112, 1920), (700, 64, 16384),
          (2304, 9216, 320), (4100, 4160, 192)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("epilogue", ["none", "gelu_tanh"])
def test_gemm(M, N, K, epilogue):
    import bit_diffusion_transformer_svdq_amd as P
    x, w = tokens(M, K, 3), weights(N, K, 3)
    if epilogue == "gelu_tanh":
        x = x[0], x[1] * np.float32(0.1)   # arguments of a few units, where GELU bends
    b = bf16(np.random.default_rng(N).standard_normal(N)) if (M + N) % 3 else None
    y = P.fp8_gemm(*_dev(x, w), dev_bf16(b), epilogue=epilogue)
    _check_gemm(host(y), x, w, b, epilogue)


@pytest.mark.parametrize("tile", [1, 114, 213, 224, 413, 423, 432, 442])
@pytest.mark.parametrize("splits", [1, 2, 16])
def test_every_tile_and_split(tile, splits):
    """The same shapes on every kernel, tile and split: one stage and less, odd numbers of
    stages, a half one at the end, ragged tokens and channels."""
    import bit_diffusion_transformer_svdq_amd as P
    for M, N, K in [(9, 64, 64), (16, 192, 192), (70, 320, 448), (300, 576, 1088), (129, 448, 2176), (129, 448, 4096), (260, 320, 960)]:
        if tile == 1 and M > 16:
            continue
        x, w = tokens(M, K, 9), weights(N, K, 9)
        b = bf16(np.random.default_rng(N).standard_normal(N))
        P.debug_set_fp8_plan(tile, splits)
        try:
            y = P.fp8_gemm(*_dev(x, w), dev_bf16(b))
        finally:
            P.debug_set_fp8_plan()
        _check_gemm(host(y), x, w, b, "none")


@pytest.mark.parametrize("M", [3, 70, 300])
@pytest.mark.parametrize("tile", [0, 114, 442])
def test_exact_sums(M, tile):
    """Codes that are small integers and scales that are powers of two: every sum is exact,
    so every block meets its own scales and every channel its own weights."""
    import bit_diffusion_transformer_svdq_amd as P
    for N, K in ((192, 448), (320, 1152)):
        g = np.random.default_rng([M, N, K])
        small = F.encode(np.arange(-4, 5).astype(float))
        x = small[g.integers(0, 9, (M, K))], 2.0 ** g.integers(-2, 3, (-(-K // 128), M)).astype(np.float32)
        w = small[g.integers(0, 9, (N, K))], 2.0 ** g.integers(-2, 3, (-(-N // 128), -(-K // 128))).astype(np.float32)
        x, w = (x[0], x[1].astype(np.float32)), (w[0], w[1].astype(np.float32))
        P.debug_set_fp8_plan(tile, 0)
        try:
            y = P.fp8_gemm(*_dev(x, w))
        finally:
            P.debug_set_fp8_plan()
        assert np.array_equal(host(y), bf16(F.product(*x, *w)[0]))


@pytest.mark.parametrize("M", [2, 300])
def test_gelu_tails(M):
    """Arguments that are exact (integers over 16), -7.5 to 7.5: the relative error is the
    function's own, (3.5 |t| + 7) 2^-24 with 2^t its exponential, and the rounding."""
    import bit_diffusion_transformer_svdq_amd as P
    v = np.concatenate([np.arange(-15, 16), np.arange(-30, 31, 2)]) / 4.0
    v = np.concatenate([v, [0.0, 0.0]])
    x, w = np.zeros((M, 64), np.uint8), np.zeros((64, 64), np.uint8)
    x[:, 5] = 0x38
    w[:, 5] = F.encode(v)
    y = host(P.fp8_gemm(dev_codes(x), dev(np.ones((1, M), np.float32)), dev_codes(w), dev(np.ones((1, 1), np.float32)),
                        epilogue="gelu_tanh"))
    u = np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
    want = v / (1 + np.exp(-2 * u))
    t = np.abs(2 * u * np.log2(np.e))
    assert (np.abs(y - want) <= (2.0 ** -8 / (1 + 2.0 ** -8) + 1.01 * (3.5 * t + 7) * U) * np.abs(want)).all()


def test_gemm_repeats_bit_for_bit_and_leaves_the_workspace_clean():
    """K-splits through one workspace, other shapes in between; the arrival counters are
    back at zero and fp32 partials are added in one order."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd import _lib
    shapes = [(130, 256, 8192), (512, 1536, 1536), (70, 64, 16384)]
    needs = [_lib.lib().svdq_fp8_gemm_workspace_size(*s) for s in shapes]
    assert any(needs)
    ws = torch.zeros(max(needs), dtype=torch.uint8, device="cuda")
    cases = [(tokens(M, K, 4), weights(N, K, 4)) for M, N, K in shapes]
    devs = [_dev(*c) for c in cases]
    first = [P.fp8_gemm(*d, workspace=ws).clone() for d in devs]
    for _ in range(5):
        for d, f in zip(devs, first):
            assert torch.equal(P.fp8_gemm(*d, workspace=ws), f)
    assert int(ws[:1 << 20].to(torch.int32).sum()) == 0
    for c, f in zip(cases, first):
        _check_gemm(host(f), *c, None, "none")


def test_runs_of_tokens():
    """Calls on a run of tokens of larger arrays, inputs and outputs, and what lies behind
    the rows stays as it was."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    K, N = 448, 192
    w = weights(N, K, 5)
    wd = dev_codes(w[0]), dev(w[1])
    for a, b in ((4, 9), (8, 140), (1, 2), (3, 19), (7, 151)):
        x, _ = acts(200, K, 5)
        codes = torch.full((200, K), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full((4, 200), 7.0, device="cuda")
        P.quantize_act_fp8(dev_bf16(x[a:b]), out=(codes[a:b], scales[:, a:b]))
        want = F.quantize_act_fp8(x[a:b])
        _same((codes[a:b], scales[:, a:b]), want)
        rest = [i for i in range(200) if not a <= i < b]
        assert (host_codes(codes)[rest] == 7).all() and (scales.cpu().numpy()[:, rest] == 7).all()
        y = torch.full((240, N), 7.0, dtype=torch.bfloat16, device="cuda")
        P.fp8_gemm(codes[a:b], scales[:, a:b], *wd, out=y[16:16 + b - a])
        _check_gemm(host(y[16:16 + b - a]), want, w, None, "none", cut=True)
        assert bool((y[:16] == 7).all()) and bool((y[16 + b - a:] == 7).all())


def test_codes_far_into_memory():
    """Rows whose codes lie beyond 4 GiB of the array's start, and scales as far."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    M, K, N = 70000, 65536, 64
    x, w = tokens(100, K, 7), weights(N, K, 7)
    codes = torch.zeros((M, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    codes[-100:].view(torch.uint8).copy_(dev(x[0]))
    wide = torch.ones((512, 4 << 20), device="cuda")   # 8 GiB
    wide[:, -100:] = dev(x[1])
    y = P.fp8_gemm(codes, wide[:, -M:], dev_codes(w[0]), dev(w[1]))
    _check_gemm(host(y[-100:]), x, w, None, "none")
    assert not bool(y[:-100].any())
    y = P.fp8_gemm(codes[-100:], wide[:, -100:], dev_codes(w[0]), dev(w[1]))
    _check_gemm(host(y), x, w, None, "none")


@pytest.mark.parametrize("M,N,K", [(2304, 9216, 448), (2560, 8192, 256), (4608, 6144, 512), (2570, 8192, 256), (4160, 12288, 192),
                                   (2050, 16384, 512), (33000, 640, 128), (3840, 12288, 320)])
def test_whole_rounds_and_the_rest(M, N, K):
    """Products of more than one round of the largest tiles run as workgroups that stay for
    several tiles, or as two launches: every row is that of one launch of a small tile, bit
    for bit (blocks are added in the order of K on every tile)."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    d = _dev(tokens(M, K, 8), weights(N, K, 8))
    b = torch.randn(N, device="cuda").bfloat16()
    y = P.fp8_gemm(*d, b)
    P.debug_set_fp8_plan(114, 1)
    try:
        one = P.fp8_gemm(*d, b)
        P.debug_set_fp8_plan(442, 1)
        big = P.fp8_gemm(*d, b)
        P.debug_set_fp8_plan(432, 1)
        mid = P.fp8_gemm(*d, b)
    finally:
        P.debug_set_fp8_plan()
    assert torch.equal(y, one) and torch.equal(big, one) and torch.equal(mid, one)


def test_packed_linear():
    """Packer, quantizer and product together against the float product."""
    import bit_diffusion_transformer_svdq_amd as P
    M, K, N = 96, 512, 320
    x, g = acts(M, K, 8)
    w = bf16(0.02 * g.standard_normal((N, K)))
    sm = np.sqrt(np.abs(x).max(0) / np.abs(w).max(0)).astype(np.float32)
    pk = P.pack_weights_fp8(O.f64_to_bf16(w), sm)
    q, s = P.quantize_act_fp8(dev_bf16(x), dev(sm))
    y = host(P.fp8_gemm(q, s, dev_codes(pk["w_codes"]), dev(pk["w_scales"])))
    xq = F.quantize_act_fp8(x, sm)
    _check_gemm(y, xq, (pk["w_codes"], pk["w_scales"]), None, "none", cut=True)
    # both quantizers round by 2^-4 of a value at most, or half a subnormal step of the scale
    xs, ws = x / sm, w * sm
    sx = np.repeat(xq[1].astype(float), 128, 0)[:K].T
    sw = np.repeat(np.repeat(pk["w_scales"].astype(float), 128, 0), 128, 1)[:N, :K]
    ex = 2.0 ** -4 * np.abs(xs) + 2.0 ** -10 * sx + 2 * HALF_BF16 * np.abs(xs)
    ew = 2.0 ** -4 * np.abs(ws) + 2.0 ** -10 * sw
    lim = ex @ np.abs(ws).T + np.abs(xs) @ ew.T + ex @ ew.T + 2 * HALF_BF16 * np.abs(xs) @ np.abs(ws).T + \
        cut_bound(*xq, pk["w_codes"], pk["w_scales"])
    assert (np.abs(y - x @ w.T) <= lim).all()
