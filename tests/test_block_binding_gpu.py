"""The block operators' binding on a device: what it refuses, whose memory a call
uses, several streams and captured graphs at once.  Needs an MI355X."""
import numpy as np
import pytest

from tests.block_util import dev

pytestmark = pytest.mark.gpu

SPLIT = (65, 128, 8192)  # few tiles, long K: K is split through the workspace


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _codes(M, N, K, seed):
    g = np.random.default_rng([seed, M, N, K])
    return (dev(g.integers(-127, 128, (M, K), dtype=np.int8)), dev((1e-2 + 1e-2 * g.random(M)).astype(np.float32)),
            dev(g.integers(-127, 128, (N, K), dtype=np.int8)), dev((1e-3 + 1e-3 * g.random(N)).astype(np.float32)))


def _plain(qx, sx, qw, sw):
    """The product from exact float64 sums; one fma and one rounding as the call's, up
    to the rounding of its int32 -> fp32 conversion."""
    return (qx.double() @ qw.double().t()) * (sx[:, None] * sw[None]).double()


def _close(y, want):
    # bf16's half step, and the conversion's and the product's fp32 ones
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all())


def _norm_args():
    import torch
    x = torch.randn(12, 128, device="cuda").bfloat16()
    return dict(x=x, y=torch.randn_like(x), gate=torch.randn(3, 128, device="cuda").bfloat16(),
                scale=torch.randn(2, 128, device="cuda").bfloat16(), shift=torch.randn(2, 128, device="cuda").bfloat16(),
                weight=torch.ones(128, device="cuda").bfloat16(), post_weight=torch.ones(128, device="cuda").bfloat16(),
                post_norm="rms")


@pytest.mark.parametrize("change,error", [
    (lambda a: dict(x=a["x"].half()), TypeError),
    (lambda a: dict(x=a["x"].t().contiguous().t()), ValueError),                 # channels not contiguous
    (lambda a: dict(y=a["y"].float()), TypeError),
    (lambda a: dict(y=a["y"][:11]), ValueError),
    (lambda a: dict(y=a["y"].cpu()), ValueError),
    (lambda a: dict(gate=a["gate"][:, :64]), ValueError),
    (lambda a: dict(gate=a["gate"].repeat(3, 1)[:5]), None),                # 5 rows do not divide 12
    (lambda a: dict(scale=a["scale"].repeat(1, 2)[:, :128]), ValueError),        # strides of scale and shift differ
    (lambda a: dict(shift=a["shift"][:1]), ValueError),
    (lambda a: dict(weight=a["weight"].float()), TypeError),
    (lambda a: dict(norm="batch"), ValueError),
    (lambda a: dict(post_norm=None), ValueError),
    (lambda a: dict(quantize="int4"), ValueError),
    (lambda a: dict(eps=float("nan")), None),
    (lambda a: dict(smooth=a["weight"].float()), None),                     # only for 8-bit output
    (lambda a: dict(h_out=a["y"]), None),                                   # an output over an input
    (lambda a: dict(h_out=a["x"].float()), TypeError),
    (lambda a: dict(out=a["x"]), None),
    (lambda a: dict(norm="none", out=a["x"].clone()), ValueError),
])
def test_norm_refusals(change, error):
    import bit_diffusion_transformer_svdq_amd as P
    args = _norm_args()
    P.gate_norm_modulate(**args)
    with pytest.raises(error or P.SvdqError):  # None: refused by the library
        P.gate_norm_modulate(**{**args, **change(args)})


def test_linear_refusals():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    qx, sx, qw, sw = _codes(20, 64, 128, 1)
    b = torch.zeros(64, device="cuda").bfloat16()
    P.w8a8_gemm(qx, sx, qw, sw, b)
    for args, error in (
            ((qx.to(torch.uint8), sx, qw, sw, b), TypeError), ((qx, sx[:19], qw, sw, b), ValueError),
            ((qx, sx, qw[:, :64], sw, b), ValueError), ((qx, sx, qw.cpu(), sw, b), ValueError),
            ((qx, sx, qw, sw.double(), b), TypeError), ((qx, sx, qw, sw, b.float()), TypeError),
            ((qx[:, ::2], sx, qw[:, ::2], sw, b), ValueError), ((qx[:, :64].contiguous()[:, :32], sx, qw, sw, b), ValueError)):
        with pytest.raises(error):
            P.w8a8_gemm(*args)
    with pytest.raises(ValueError):
        P.w8a8_gemm(qx, sx, qw, sw, b, epilogue="relu")
    with pytest.raises(ValueError):
        P.w8a8_gemm(qx, sx, qw, sw, b, out=torch.empty(20, 65, device="cuda").bfloat16())
    with pytest.raises(P.SvdqError):   # a workspace that is too small
        P.w8a8_gemm(*_codes(*SPLIT, 1), workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(20, 128, device="cuda").bfloat16()
    for args, error in (((x.float(),), TypeError), ((x[:, ::2],), ValueError),
                        ((x, torch.ones(64, device="cuda")), ValueError), ((x, torch.ones(128)), ValueError)):
        with pytest.raises(error):
            P.quantize_act_int8(*args)


def test_rope_refusals():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    q = torch.randn(12, 2, 128, device="cuda").bfloat16()
    k = torch.randn(12, 1, 128, device="cuda").bfloat16()
    pos = torch.zeros(6, 3, dtype=torch.int32, device="cuda")
    axes, w = (16, 56, 56), torch.ones(128, device="cuda").bfloat16()
    P.rope_axes(q, k, pos, axes, q_norm=w, k_norm=w)
    for args, kw, error in (
            ((q.float(), k, pos, axes), {}, TypeError), ((q, k[:11], pos, axes), {}, ValueError),
            ((q, k, pos.long(), axes), {}, TypeError), ((q, k, pos[:5], axes), {}, P.SvdqError),
            ((q, k, pos, (16, 56)), {}, ValueError), ((q, k, pos, (16, 56, 58)), {}, P.SvdqError),
            ((q, k, pos.cpu(), axes), {}, ValueError), ((q.transpose(0, 1), None, pos, axes), {}, ValueError),
            ((q, k, pos, axes), dict(q_norm=w), P.SvdqError), ((q, k, pos, axes), dict(layout="rows"), ValueError),
            ((q, k, pos, axes), dict(spectrum="one"), ValueError), ((q, k, pos, axes), dict(theta=1.0), P.SvdqError),
            ((q, k, pos, axes), dict(out=(torch.empty_like(q), None)), ValueError),
            ((q, k, pos, axes), dict(out=(q, q[:, :1])), P.SvdqError)):
        with pytest.raises(error):
            P.rope_axes(*args, **kw)
    with pytest.raises(TypeError):
        P.rope_axes_tables(pos.double(), axes)
    with pytest.raises(P.SvdqError):
        P.rope_axes_tables(pos, (16, 57, 55))


def test_given_outputs_are_kept_for_the_stream():
    """An output freed right after a call on another stream is not handed out again
    while that stream may still write it."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    x = torch.randn(64, 4096, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = (torch.empty(64, 4096, dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda"))
    at = out[0].data_ptr()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    P.quantize_act_int8(x, out=out, stream=s)
    busy = not s.query()
    del out
    again = torch.empty(64, 4096, dtype=torch.int8, device="cuda")
    assert again.data_ptr() != at or not busy
    torch.cuda.synchronize()


def test_split_products_on_two_streams_at_once():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd import _lib
    assert _lib.lib().svdq_w8a8_gemm_workspace_size(*SPLIT) > 0
    cases = [_codes(*SPLIT, seed) for seed in (2, 3)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                g.append(P.w8a8_gemm(*c))
    torch.cuda.synchronize()
    for c, g in zip(cases, got):
        _close(g[0], _plain(*c))
        assert all(torch.equal(t, g[0]) for t in g)


def test_graphs_captured_on_one_stream_replayed_on_two():
    """Each graph has a workspace of its own: replays side by side, and beside eager
    calls that split K too, give the eager results."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    cases = [_codes(*SPLIT, seed) for seed in (4, 5, 6)]
    want = [P.w8a8_gemm(*c).clone() for c in cases]
    for c, w in zip(cases, want):
        _close(w, _plain(*c))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for c in cases[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            ys = [P.w8a8_gemm(*c) for _ in range(4)]
        graphs.append((g, ys))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for _, ys in graphs:
            for y in ys:
                y.fill_(7)
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [P.w8a8_gemm(*cases[2]) for _ in range(4)]
        torch.cuda.synchronize()
        for (_, ys), w in zip(graphs, want):
            assert all(torch.equal(y, w) for y in ys)
        assert all(torch.equal(y, want[2]) for y in eager)


def test_capture_with_a_stream_argument():
    """The stream given by hand is the one being captured."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    c = _codes(*SPLIT, 7)
    want = P.w8a8_gemm(*c).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = P.w8a8_gemm(*c, stream=torch.cuda.current_stream())
    for _ in range(3):
        y.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [(2570, 8192, 256), (4160, 12288, 192), (2050, 16384, 512), (33000, 640, 128)])
@pytest.mark.parametrize("epilogue", ["none", "gelu_tanh"])
def test_whole_rounds_and_the_rest(M, N, K, epilogue):
    """Products of more than one round of the large tile run as two launches; every
    row is that of one launch of a small tile (sums of integers)."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    c = _codes(M, N, K, 8)
    b = torch.randn(N, device="cuda").bfloat16()
    y = P.w8a8_gemm(*c, b, epilogue=epilogue)
    P.debug_set_w8a8_plan(114, 1)
    try:
        one = P.w8a8_gemm(*c, b, epilogue=epilogue)
    finally:
        P.debug_set_w8a8_plan()
    assert torch.equal(y, one)
    rows = [0, 1, M // 2, M - 40, M - 1]
    if epilogue == "none":
        want = _plain(c[0][rows], c[1][rows], c[2], c[3]) + b.double()
        err = (2.0 ** -8 + 2.0 ** -20) * want.abs() + 2.0 ** -22 * (want - b.double()).abs()
        assert bool(((y[rows].double() - want).abs() <= err).all())


@pytest.mark.parametrize("tile,M,N,K", [(442, 1024, 16640, 256), (442, 256, 65792, 512), (442, 256, 131328, 256),
                                        (342, 1536, 10752, 768), (432, 4032, 6656, 256), (432, 384, 65536, 1024),
                                        (442, 1025, 16640, 256), (442, 1024, 16640, 320), (442, 1024, 16576, 384)])
def test_many_tiles_per_workgroup(tile, M, N, K):
    """Whole tiles, more of them than compute units and by one or two only: a
    workgroup's first and last tile come out as in a launch of small tiles; and what
    is not whole (rows, channels, stages)."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    c = _codes(M, N, K, 9)
    b = torch.randn(N, device="cuda").bfloat16()
    got = []
    for t in (tile, 124):
        P.debug_set_w8a8_plan(t, 1)
        try:
            got.append([P.w8a8_gemm(*c, b, epilogue=e) for e in ("none", "gelu_tanh")])
        finally:
            P.debug_set_w8a8_plan()
    for y, w in zip(*got):
        assert torch.equal(y, w)
