"""The gated feed-forward product (svdq_fp8_gated_gemm), the norms that write e4m3 codes and
the feed-forward block that they make up, against the oracle.  Needs an MI355X.  Bounds:
tests/fp8_util.py; a code is off by at most half its step from a value that the fp32
arithmetic knows up to its bound."""
import numpy as np
import pytest

import oracle as O
import oracle.block_oracle as B
import oracle.fp8_oracle as F
from tests.block_util import HALF_BF16, SLACK, U, bf16, check, dev, dev_bf16, gate_norm_bound, host
from tests.fp8_util import acts, cut_bound, dev_codes, gated_bound, host_codes, product_bound, tokens, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _case(M, N, K, seed, bias=True):
    x, gate, up = tokens(M, K, seed), weights(N, K, seed), weights(N, K, seed + 100)
    g = np.random.default_rng([seed, M, N, K, 3])
    x = x[0], x[1] * np.float32(0.2)   # gate arguments of a few units
    b = [bf16(0.3 * g.standard_normal(N)) if bias else None for _ in range(2)]
    return x, gate, up, b


def _call(x, gate, up, b, **kw):
    import bit_diffusion_transformer_svdq_amd as P
    return P.fp8_gated_gemm(dev_codes(x[0]), dev(x[1]), dev_codes(gate[0]), dev(gate[1]), dev_codes(up[0]), dev(up[1]),
                            dev_bf16(b[0]), dev_bf16(b[1]), **kw)


def check_codes(codes, scales, v, ev):
    """Codes and scales of values v known up to ev."""
    M, N = v.shape
    pad = -N % 128
    blocks = np.pad(np.abs(v), ((0, 0), (0, pad))).reshape(M, -1, 128)
    eb = np.pad(ev, ((0, 0), (0, pad))).reshape(M, -1, 128)
    s = scales.astype(float).T
    assert (s <= (blocks + eb).max(2) / 448 * (1 + 4 * U) + 1e-44).all()
    assert (s >= (blocks - eb).max(2).clip(0) / 448 * (1 - 4 * U) - 1e-44).all()
    wide = np.repeat(s, 128, 1)[:, :N]
    step = np.maximum(2.0 ** -4 * (np.abs(v) + ev), 2.0 ** -10 * wide)  # half a step, of a code or below the least
    lim = SLACK * (ev + step + 8 * U * np.abs(v)) + 1e-38
    assert (np.abs(F.decode(codes) * wide - v) <= lim).all()


def _check_out(got, x, gate, up, b, act, smooth=None, cut=False):
    h, eh = gated_bound(*x, gate, up, *b, act, cut=cut)
    if not isinstance(got, tuple):
        check(host(got), h, eh)
        return
    if smooth is not None:
        h, eh = h / smooth, eh / smooth + 2 * U * np.abs(h / smooth)
    check_codes(host_codes(got[0]), got[1].cpu().numpy(), h, eh)


SHAPES = [(1, 64, 64), (1, 1536, 1536), (2, 192, 320), (16, 128, 1024), (16, 4160, 192), (5, 64, 16384), (9, 320, 448),
          (17, 1088, 192), (33, 64, 8192), (64, 4160, 576), (65, 128, 192), (127, 320, 640), (257, 576, 448),
          (512, 1024, 1088), (1333, 2112, 960), (2304, 4608, 320), (4100, 4160, 192)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated(M, N, K, act):
    c = _case(M, N, K, 1, bias=(M + N) % 3 > 0)
    _check_out(_call(*c, activation=act), *c, act)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("smooth", [False, True])
def test_gated_codes(M, N, K, smooth):
    c = _case(M, N, K, 2, bias=(M + N) % 3 > 0)
    sm = np.exp(0.7 * np.random.default_rng(N).standard_normal(N)).astype(np.float32) if smooth else None
    got = _call(*c, quantize="fp8", smooth=None if sm is None else dev(sm))
    assert got[1].shape == (-(-N // 128), M)
    _check_out(got, *c, "silu", sm)


@pytest.mark.parametrize("tile", [1, 114, 213, 224, 413, 423, 432, 442])
@pytest.mark.parametrize("splits", [1, 2, 16])
@pytest.mark.parametrize("quantize", [None, "fp8"])
def test_every_tile_and_split(tile, splits, quantize):
    import bit_diffusion_transformer_svdq_amd as P
    for M, N, K in [(9, 64, 64), (16, 192, 192), (70, 320, 448), (300, 576, 1088), (129, 448, 2176), (260, 320, 960)]:
        if tile == 1 and M > 16:
            continue
        c = _case(M, N, K, 9)
        P.debug_set_fp8_plan(tile, splits)
        try:
            got = _call(*c, quantize=quantize)
        finally:
            P.debug_set_fp8_plan()
        _check_out(got, *c, "silu")


@pytest.mark.parametrize("M,N,K", [(2304, 4608, 192), (2560, 4096, 512), (3840, 4096, 256), (2570, 4160, 256), (4100, 6144, 192), (2050, 8192, 448)])
@pytest.mark.parametrize("quantize", [None, "fp8"])
def test_whole_rounds_and_the_rest(M, N, K, quantize):
    """As for the plain product, bf16 against a small tile, codes against the smallest that
    holds a block of features; codes of some tokens against the oracle."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    c = _case(M, N, K, 8)

    def bits():
        r = _call(*c, quantize=quantize)
        return [t.view(torch.uint8) for t in (r if isinstance(r, tuple) else (r,))], r
    got, out = bits()
    for tile in (413 if quantize else 114, 432, 442):
        P.debug_set_fp8_plan(tile, 1)
        try:
            want, _ = bits()
        finally:
            P.debug_set_fp8_plan()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), tile
    rows = np.unique(np.concatenate([np.arange(0, M, 97), [M - 1]]))
    part = (c[0][0][rows], c[0][1][:, rows]), *c[1:]
    at = torch.from_numpy(rows).cuda()
    some = out[at] if quantize is None else (out[0].view(torch.uint8)[at].view(torch.float8_e4m3fn), out[1][:, at])
    _check_out(some, *part, "silu")


@pytest.mark.parametrize("M", [3, 16, 70, 300])
@pytest.mark.parametrize("N", [64, 128, 448])
def test_exact_codes(M, N):
    """Gates of 64 (SiLU gives 64 itself: exp(-64) is lost in 1 + exp(-64)) and whole numbers
    for U: H is exact, so its codes and scales are those of the quantizer."""
    import bit_diffusion_transformer_svdq_amd as P
    K = 192
    g = np.random.default_rng([M, N])
    x = np.zeros((M, K), np.uint8), np.ones((2, M), np.float32)
    x[0][:, 0] = 0x38
    x[0][:, 1:] = F.encode(np.arange(-2, 3).astype(float))[g.integers(0, 5, (M, K - 1))]
    gate = np.zeros((N, K), np.uint8), np.ones((-(-N // 128), 2), np.float32)
    gate[0][:, 0] = F.encode(64.0)
    up = F.encode(np.arange(-4, 5).astype(float))[g.integers(0, 9, (N, K))], np.ones((-(-N // 128), 2), np.float32)
    h = 64 * F.product(*x, *up)[0]
    h[0] = 0 if M == 3 else h[0]
    if M == 3:
        x[0][0, 1:] = 0
        up[0][:, 0] = 0
        h = 64 * F.product(*x, *up)[0]
        assert not h[0].any()          # a row of zeros: codes 0, scales 0
    sm = (2.0 ** g.integers(-2, 3, N)).astype(np.float32)
    for s in (None, sm):
        want = F.quantize(h if s is None else h / s)
        got = _call(x, gate, up, (None, None), quantize="fp8", smooth=None if s is None else dev(s))
        assert np.array_equal(got[1].cpu().numpy(), want[1])
        # (the sign of a zero is not fixed: H may be the product of -0)
        assert np.array_equal(F.decode(host_codes(got[0])), F.decode(want[0]))
    assert np.array_equal(host(_call(x, gate, up, (None, None))), bf16(h))
    assert P is not None


@pytest.mark.parametrize("M", [4, 90])
def test_bad_tokens_stay_alone(M):
    """A NaN scale of one token, and an overflow to infinity: rows of NaN or infinity,
    or codes 0 with NaN scales, and no other row is touched."""
    x, gate, up, b = _case(M, 320, 192, 5)
    x[1][1, 2] = np.nan
    x[1][:, 3] = 3e38
    with np.errstate(all="ignore"):
        good = np.delete(np.arange(M), (2, 3))
        c = (x[0][good], x[1][:, good]), gate, up, b
    y = host(_call(x, gate, up, b))
    assert np.isnan(y[2]).all() and not np.isfinite(y[3]).all()
    h, eh = gated_bound(*c[0], gate, up, *b, "silu")
    check(y[good], h, eh)
    q, s = _call(x, gate, up, b, quantize="fp8")
    s = s.cpu().numpy()
    assert np.isnan(s[:, 2]).all() and not host_codes(q)[2].any() and np.isnan(s[:, 3]).any()
    check_codes(host_codes(q)[good], s[:, good], h, eh)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [2, 100])
def test_activation_tails(act, M):
    """Gates that are exact (-60 to 60) times an exact 1: the relative error is the
    function's own ((|x| + 5) 2^-24 for SiLU, (3.5 |t| + 7) 2^-24 for GELU above -10) and
    the rounding."""
    v = np.concatenate([np.arange(-15, 16) * 4.0, np.arange(-15, 16) / 2.0, [0.0, 0.0]])
    if act == "gelu_tanh":
        v = np.clip(v, -7.5, 60)
    x = np.zeros((M, 64), np.uint8), np.ones((1, M), np.float32)
    x[0][:, 7] = 0x38
    gate = np.zeros((64, 64), np.uint8), np.ones((1, 1), np.float32)
    gate[0][:, 7] = F.encode(v)
    up = np.zeros((64, 64), np.uint8), np.ones((1, 1), np.float32)
    up[0][:, 7] = 0x38
    y = host(_call(x, gate, up, (None, None), activation=act))
    if act == "silu":
        want, own = v / (1 + np.exp(-v)), (np.abs(v) + 5) * U
    else:
        u = np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        want, own = v / (1 + np.exp(-2 * u)), (3.5 * np.abs(2 * u * np.log2(np.e)) * (v < 0) + 7) * U
    assert (np.abs(y - want) <= (2.0 ** -8 / (1 + 2.0 ** -8) + 1.01 * own) * np.abs(want) + 1e-38).all()


def test_repeats_bit_for_bit_and_leaves_the_workspace_clean():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd import _lib
    shapes = [(130, 256, 8192, None), (16, 4160, 1536, "fp8"), (70, 64, 8192, "fp8"), (3, 192, 320, "fp8"), (70, 64, 8192, None)]
    kind = {None: 0, "fp8": 1}
    needs = [_lib.lib().svdq_fp8_gated_gemm_workspace_size(M, N, K, kind[q]) for M, N, K, q in shapes]
    assert needs[1] and needs[2] and needs[3]
    ws = torch.zeros(max(needs), dtype=torch.uint8, device="cuda")
    cases = [_case(M, N, K, 4) for M, N, K, _ in shapes]

    def bits(i):
        r = _call(*cases[i], quantize=shapes[i][3], workspace=ws)
        return [t.clone().view(torch.uint8) for t in (r if isinstance(r, tuple) else (r,))]
    first = [bits(i) for i in range(len(shapes))]
    for _ in range(4):
        for i, f in enumerate(first):
            assert all(torch.equal(a, b) for a, b in zip(bits(i), f))
    assert int(ws[:1 << 20].to(torch.int32).sum()) == 0
    assert P is not None


def test_leaves_what_is_behind_its_rows():
    import torch
    for M in (5, 130):
        c = _case(M, 192, 256, 6)
        buf = torch.full((M + 40, 192), 7.0, dtype=torch.bfloat16, device="cuda")
        _call(*c, out=buf[:M])
        assert bool((buf[M:] == 7).all())
        codes = torch.full((M + 40, 192), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full((3, M + 40), 7.0, device="cuda")
        _call(*c, quantize="fp8", out=(codes[:M], scales[:2, :M]))
        assert (host_codes(codes[M:]) == 7).all() and bool((scales[:, M:] == 7).all()) and bool((scales[2] == 7).all())
        _check_out((codes[:M], scales[:2, :M]), *c, "silu")


# ------------------------------------------------------------- norms into codes

def _norm_case(M, B_, C, seed, fp32=False):
    g = np.random.default_rng([seed, M, C])
    x = g.standard_normal((M, C)) * 3
    x = x.astype(np.float32).astype(float) if fp32 else bf16(x)
    return dict(x=x, y=bf16(g.standard_normal((M, C))), gate=bf16(g.standard_normal((B_, C))), scale=bf16(0.3 * g.standard_normal((B_, C))),
                shift=bf16(0.3 * g.standard_normal((B_, C))), weight=bf16(1 + 0.1 * g.standard_normal(C)),
                post_weight=bf16(1 + 0.1 * g.standard_normal(C)), post_norm="rms"), np.exp(0.5 * g.standard_normal(C)).astype(np.float32)


@pytest.mark.parametrize("M,B_,C", [(1, 1, 64), (3, 3, 192), (6, 2, 576), (4, 1, 1536), (40, 2, 2304), (600, 3, 1088), (9, 1, 4160), (4, 2, 8256),
                                    (3, 1, 16448), (2, 1, 32768), (2100, 1, 1024), (520, 2, 4096)])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("smooth", [False, True])
def test_norm_codes(M, B_, C, fp32, smooth):
    import bit_diffusion_transformer_svdq_amd as P
    a, sm = _norm_case(M, B_, C, 1, fp32)
    kind = "layer" if C % 3 else "rms"
    kw = {k: (v if isinstance(v, str) else dev_bf16(v)) for k, v in a.items() if k != "x"}
    x = dev(a["x"].astype(np.float32)) if fp32 else dev_bf16(a["x"])
    h, (q, s) = P.gate_norm_modulate(x, norm=kind, quantize="fp8", smooth=dev(sm) if smooth else None, **kw)
    wh, eh, z, ez = gate_norm_bound(**a, norm=kind)
    check(host(h), wh, eh, half=U if fp32 else HALF_BF16)
    if smooth:
        z, ez = z / sm, ez / sm + 2 * U * np.abs(z / sm)
    assert s.shape == (-(-C // 128), M)
    check_codes(host_codes(q), s.cpu().numpy(), z, ez)


def test_norm_codes_are_those_of_the_quantizer():
    """RMS norm of rows of one magnitude, all powers of two: z is exact, so its codes and
    scales are the quantizer's; a zero row, and rows with infinities and NaN beside it."""
    import bit_diffusion_transformer_svdq_amd as P
    C, M = 320, 7
    g = np.random.default_rng(3)
    x = np.where(g.random((M, C)) < 0.5, -4.0, 4.0)
    scale = bf16((2.0 ** g.integers(-3, 4, (1, C))) - 1)
    x[3] = 0
    h, (q, s) = P.gate_norm_modulate(dev_bf16(x), norm="rms", eps=0.0, scale=dev_bf16(scale), quantize="fp8")
    want = F.quantize(np.sign(np.delete(x, 3, 0)) * (1 + scale))
    keep = np.delete(np.arange(M), 3)
    assert h is None
    assert np.array_equal(host_codes(q)[keep], want[0]) and np.array_equal(s.cpu().numpy()[:, keep], want[1])
    assert np.isnan(s.cpu().numpy()[:, 3]).all()            # 0 / 0
    h, (q0, s0) = P.gate_norm_modulate(dev_bf16(x), norm="rms", eps=1e-6, quantize="fp8")
    assert not host_codes(q0)[3].any() and not s0.cpu().numpy()[:, 3].any()
    y = x.copy()
    y[1, 5], y[2, 300] = np.inf, np.nan
    _, (q1, s1) = P.gate_norm_modulate(dev_bf16(y), norm="rms", eps=1e-6, quantize="fp8")
    rest = [0, 3, 4, 5, 6]
    assert np.array_equal(host_codes(q1)[rest], host_codes(q0)[rest]) and not host_codes(q1)[2].any()
    assert np.isnan(s1.cpu().numpy()[:, 2]).all() and np.isnan(s1.cpu().numpy()[0, 1])


def test_norm_codes_on_other_calls_results():
    """The int8 and bf16 outputs of the same call are what they were beside it."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    a, sm = _norm_case(70, 2, 1088, 4)
    kw = {k: (v if isinstance(v, str) else dev_bf16(v)) for k, v in a.items()}
    h0, z = P.gate_norm_modulate(**kw)
    h1, (q8, s8) = P.gate_norm_modulate(**kw, quantize="int8")
    h2, (q, s) = P.gate_norm_modulate(**kw, quantize="fp8")
    assert torch.equal(h0, h1) and torch.equal(h0, h2)
    _, _, want, ez = gate_norm_bound(**a)
    check(host(z), want, ez)
    assert np.abs(q8.cpu().numpy() * s8.cpu().numpy()[:, None] - want).max() <= 0.51 * s8.max().item()
    check_codes(host_codes(q), s.cpu().numpy(), want, ez)


# ----------------------------------------------------------------- the whole block

def _ffn(M, K, Fc, seed, bias=True):
    """The packed layers of a block, on the host, and its input."""
    import bit_diffusion_transformer_svdq_amd as P
    x, g = acts(M, K, seed)
    sm = np.sqrt(np.abs(x).max(0).clip(1e-2) / 0.08).astype(np.float32)
    smh = np.exp(0.5 * g.standard_normal(Fc)).astype(np.float32)
    out = []
    for N, k, s in ((Fc, K, sm), (Fc, K, sm), (K, Fc, smh)):
        p = P.pack_weights_fp8(O.f64_to_bf16(0.02 * g.standard_normal((N, k))), s)
        out.append(dict(w_codes=p["w_codes"], w_scales=p["w_scales"], smooth=s, bias=bf16(0.05 * g.standard_normal(N)) if bias else None))
    return x, out


def _to_dev(layer):
    return dict(w_codes=dev_codes(layer["w_codes"]), w_scales=dev(layer["w_scales"]), smooth=dev(layer["smooth"]),
                bias=dev_bf16(layer["bias"]))


def _w(layer):
    return layer["w_codes"], layer["w_scales"]


@pytest.mark.parametrize("M,K,Fc", [(1, 192, 320), (16, 256, 704), (77, 576, 1088), (300, 320, 640)])
def test_whole_block(M, K, Fc):
    """Quantizer, gated product and down-projection, one after the other, each against the
    oracle on what it was given, and the block's call, which must be the same three."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    x, (gate, up, down) = _ffn(M, K, Fc, 7)
    gd, ud, dd = map(_to_dev, (gate, up, down))
    q, s = P.quantize_act_fp8(dev_bf16(x), gd["smooth"])
    xq = F.quantize_act_fp8(x, gate["smooth"])
    assert np.array_equal(host_codes(q), xq[0]) and np.array_equal(s.cpu().numpy(), xq[1])
    hq = P.fp8_gated_gemm(q, s, gd["w_codes"], gd["w_scales"], ud["w_codes"], ud["w_scales"], gd["bias"], ud["bias"],
                          quantize="fp8", smooth=dd["smooth"])
    _check_out(hq, xq, _w(gate), _w(up), (gate["bias"], up["bias"]), "silu", down["smooth"], cut=True)
    y = P.fp8_gemm(*hq, dd["w_codes"], dd["w_scales"], dd["bias"])
    given = host_codes(hq[0]), hq[1].cpu().numpy()
    v, mags = F.product(*given, *_w(down), down["bias"])
    check(host(y), v, product_bound(Fc, mags, v) + cut_bound(*given, *_w(down)))
    again = P.gated_ffn_fp8(dev_bf16(x), gd, ud, dd)
    assert torch.equal(again, y)
    # and the float block: quantizing both inputs and all weights leaves about 2^-4 of each
    # term, which adds up like noise; no bound, but a wrong scale or layer would show
    w = [F.weight_values(*_w(t)) for t in (gate, up, down)]
    xs = x / gate["smooth"]
    h = F.silu(xs @ w[0].T + gate["bias"]) * (xs @ w[1].T + up["bias"]) / down["smooth"]
    ref = h @ w[2].T + down["bias"]
    assert np.linalg.norm(host(y) - ref) <= 0.15 * np.linalg.norm(ref)


def test_norm_block_chain():
    """The norm's codes straight into the gated product, as a block runs them."""
    import bit_diffusion_transformer_svdq_amd as P
    M, C, Fc = 90, 576, 640
    a, _ = _norm_case(M, 2, C, 8)
    _, (gate, up, down) = _ffn(M, C, Fc, 9)
    gd, ud, dd = map(_to_dev, (gate, up, down))
    kw = {k: (v if isinstance(v, str) else dev_bf16(v)) for k, v in a.items()}
    h, (q, s) = P.gate_norm_modulate(**kw, quantize="fp8", smooth=gd["smooth"])
    given = host_codes(q), s.cpu().numpy()
    out = P.fp8_gated_gemm(q, s, gd["w_codes"], gd["w_scales"], ud["w_codes"], ud["w_scales"], gd["bias"], ud["bias"],
                           activation="gelu_tanh")
    _check_out(out, given, _w(gate), _w(up), (gate["bias"], up["bias"]), "gelu_tanh", cut=True)
    _, _, z, ez = gate_norm_bound(**a)
    check_codes(*given, z / gate["smooth"], ez / gate["smooth"] + 2 * U * np.abs(z / gate["smooth"]))
    assert B is not None
