"""The 8-bit floating-point linear's binding on a device: what it refuses, whose memory a
call uses, several streams and captured graphs at once.  Needs an MI355X."""
import numpy as np
import pytest

from tests.block_util import dev, dev_bf16, host
from tests.fp8_util import acts, dev_codes, tokens, weights

pytestmark = pytest.mark.gpu

SPLIT = (65, 128, 8192)    # few tiles, long K: K is split through the workspace
FEW = (7, 1088, 1536)      # few tokens into codes: blocks of features meet in the workspace


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _args(M, N, K, seed):
    x, w = tokens(M, K, seed), weights(N, K, seed)
    return dev_codes(x[0]), dev(x[1]), dev_codes(w[0]), dev(w[1])


def _gated(M, N, K, seed):
    u = weights(N, K, seed + 50)
    return *_args(M, N, K, seed), dev_codes(u[0]), dev(u[1])


def _bits(r):
    import torch
    return [t.contiguous().view(torch.uint8) for t in (r if isinstance(r, tuple) else (r,))]


def _calls(seed):
    """One call of each kind that goes through a workspace, as functions of nothing."""
    import bit_diffusion_transformer_svdq_amd as P
    a, b, c = _args(*SPLIT, seed), _gated(*SPLIT, seed), _gated(*FEW, seed)
    return [lambda **kw: P.fp8_gemm(*a, **kw), lambda **kw: P.fp8_gated_gemm(*b, quantize="fp8", **kw),
            lambda **kw: P.fp8_gated_gemm(*c, quantize="fp8", **kw)]


def test_the_calls_use_a_workspace():
    from bit_diffusion_transformer_svdq_amd import _lib
    assert _lib.lib().svdq_fp8_gemm_workspace_size(*SPLIT) > 0
    assert _lib.lib().svdq_fp8_gated_gemm_workspace_size(*SPLIT, 1) > 0
    assert _lib.lib().svdq_fp8_gated_gemm_workspace_size(*FEW, 1) > 0


def test_refusals():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    M, N, K = 20, 192, 320
    q, s, w, z, u, v = _gated(M, N, K, 1)
    b = torch.zeros(N, device="cuda").bfloat16()
    P.fp8_gemm(q, s, w, z, b)
    P.fp8_gated_gemm(q, s, w, z, u, v, b, b)
    for args, error in (
            ((q.view(torch.uint8), s, w, z, b), TypeError), ((q, s[:, :19], w, z, b), ValueError), ((q, s[:2], w, z, b), ValueError),
            ((q, s.t().contiguous().t(), w, z, b), ValueError),                   # tokens not contiguous
            ((q, s, w[:, :64], z, b), ValueError), ((q, s, w.cpu(), z, b), ValueError), ((q, s, w, z[:1], b), ValueError),
            ((q, s, w, z.double(), b), TypeError), ((q, s, w, z, b.float()), TypeError), ((q[:, ::2], s, w, z, b), ValueError),
            ((q, s.bfloat16(), w, z, b), TypeError), ((q, s[:1].expand(3, M), w, z, b), P.SvdqError)):   # stride 0
        with pytest.raises(error):
            P.fp8_gemm(*args)
        with pytest.raises(error):
            P.fp8_gated_gemm(*args[:4], u, v, args[4])
    for kw, error in ((dict(epilogue="relu"), ValueError), (dict(out=torch.empty(20, 65, device="cuda").bfloat16()), ValueError),
                      (dict(out=torch.empty(20, N, device="cuda")), TypeError)):
        with pytest.raises(error):
            P.fp8_gemm(q, s, w, z, b, **kw)
    for kw, error in ((dict(activation="relu"), ValueError), (dict(quantize="int8"), ValueError), (dict(up_bias=b[:64]), ValueError),
                      (dict(smooth=torch.ones(N, device="cuda")), P.SvdqError), (dict(smooth=b, quantize="fp8"), TypeError),
                      (dict(out=(q, s), quantize="fp8"), ValueError), (dict(out=torch.empty(20, N, device="cuda")), TypeError)):
        with pytest.raises(error):
            P.fp8_gated_gemm(q, s, w, z, u, v, **kw)
    for call in (lambda ws: P.fp8_gemm(*_args(*SPLIT, 1), workspace=ws),
                 lambda ws: P.fp8_gated_gemm(*_gated(*FEW, 1), quantize="fp8", workspace=ws)):
        with pytest.raises(P.SvdqError):   # a workspace that is too small
            call(torch.zeros(64, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(20, 128, device="cuda").bfloat16()
    for args, kw, error in (((x.float(),), {}, TypeError), ((x[:, ::2],), {}, ValueError), ((x[:, :96].contiguous(),), {}, P.SvdqError),
                            ((x, torch.ones(64, device="cuda")), {}, ValueError), ((x, torch.ones(128)), {}, ValueError),
                            ((x,), dict(out=(x, s)), TypeError),
                            ((x,), dict(out=(q[:, :128].contiguous(), torch.empty(2, 20, device="cuda"))), ValueError)):
        with pytest.raises(error):
            P.quantize_act_fp8(*args, **kw)
    with pytest.raises(ValueError):
        P.gate_norm_modulate(x, quantize="fp16")
    with pytest.raises(P.SvdqError):
        P.gate_norm_modulate(x, norm="none", quantize="fp8")


def test_no_rows():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    q, s, w, z, u, v = _gated(20, 192, 320, 1)
    x = torch.zeros(0, 320, device="cuda").bfloat16()
    c, t = P.quantize_act_fp8(x)
    assert c.shape == (0, 320) and t.shape == (3, 0)
    assert P.fp8_gemm(c, t, w, z).shape == (0, 192) and P.fp8_gated_gemm(c, t, w, z, u, v).shape == (0, 192)
    c, t = P.fp8_gated_gemm(c, t, w, z, u, v, quantize="fp8")
    assert c.shape == (0, 192) and t.shape == (2, 0)


def test_given_outputs_are_kept_for_the_stream():
    """An output freed right after a call on another stream is not handed out again
    while that stream may still write it."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    x = dev_bf16(acts(64, 4096, 1)[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = (torch.empty(64, 4096, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.empty(32, 64, device="cuda"))
    at = out[0].data_ptr()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    P.quantize_act_fp8(x, out=out, stream=s)
    busy = not s.query()
    del out
    again = torch.empty(64, 4096, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != at or not busy
    torch.cuda.synchronize()


def test_products_on_two_streams_at_once():
    import torch
    cases = [_calls(seed) for seed in (2, 3)]
    want = [[_bits(f()) for f in c] for c in cases]
    want = [[[t.clone() for t in r] for r in c] for c in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                g.append([_bits(f()) for f in c])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for rs in g:
            assert all(torch.equal(a, b) for r, x in zip(rs, w) for a, b in zip(r, x))


def test_graphs_captured_on_one_stream_replayed_on_two():
    """Each graph has workspaces of its own: replays side by side, and beside eager calls,
    give the eager results."""
    import torch
    cases = [_calls(seed) for seed in (4, 5, 6)]
    want = [[[t.clone() for t in _bits(f())] for f in c] for c in cases]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for c in cases[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            rs = [f() for f in c for _ in range(2)]
        graphs.append((g, rs))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for _, rs in graphs:
            for r in rs:
                for t in _bits(r):
                    t.fill_(7)
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [f() for f in cases[2]]
        torch.cuda.synchronize()
        for (_, rs), w in zip(graphs, want):
            for i, r in enumerate(rs):
                assert all(torch.equal(a, b) for a, b in zip(_bits(r), w[i // 2]))
        for r, w in zip(eager, want[2]):
            assert all(torch.equal(a, b) for a, b in zip(_bits(r), w))


def test_a_captured_block_follows_its_inputs():
    """The whole block captured with a stream given by hand, replayed on new inputs."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    K, Fc = 576, 1088
    for M in (7, 90):
        layers = []
        for i, (n, k) in enumerate(((Fc, K), (Fc, K), (K, Fc))):
            w = weights(n, k, 20 + i)
            layers.append(dict(w_codes=dev_codes(w[0]), w_scales=dev(w[1]), bias=None, smooth=torch.full((k,), 1.5, device="cuda")))
        xs = [dev_bf16(acts(M, K, seed)[0]) for seed in (1, 2, 3)]
        want = [P.gated_ffn_fp8(x, *layers).clone() for x in xs]
        x = xs[0].clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            y = P.gated_ffn_fp8(x, *layers, stream=torch.cuda.current_stream())
        for i in (1, 2, 0, 1):
            x.copy_(xs[i])
            y.fill_(7)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i])
            P.gated_ffn_fp8(xs[2], *layers)


def test_a_call_on_another_stream():
    """stream=: the call's work, outputs and workspace belong to that stream."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    s = torch.cuda.Stream()
    for f in _calls(9):
        want = [t.clone() for t in _bits(f())]
        torch.cuda.synchronize()
        got = f(stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_bits(got), want))
    x = dev_bf16(acts(40, 320, 3)[0])
    want = P.quantize_act_fp8(x)
    torch.cuda.synchronize()
    got = P.quantize_act_fp8(x, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(_bits(got), _bits(want)))
    assert np.isfinite(host(got[1])).all()
