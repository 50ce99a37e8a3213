"""The block operators together, as a transformer block runs them: eagerly, in a
captured graph and on another stream.  Needs an MI355X."""
import numpy as np
import pytest

import oracle as O
import oracle.block_oracle as B
from tests.block_util import bf16, dev, dev_bf16, host

pytestmark = pytest.mark.gpu

M, C, HEADS, AXES, HID = 130, 256, 2, (16, 56, 56), 512


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


@pytest.fixture(scope="module")
def block():
    import bit_diffusion_transformer_svdq_amd as P
    g = np.random.default_rng(17)
    w = {}
    for name, n, k in (("qkv", 3 * HEADS * 128, C), ("up", HID, C), ("down", C, HID)):
        sm = np.exp(0.3 * g.standard_normal(k)).astype(np.float32)
        pk = P.pack_weights_int8(O.f64_to_bf16(0.05 * g.standard_normal((n, k))), sm)
        w[name] = (sm, pk["w_codes"], pk["w_scales"], bf16(0.1 * g.standard_normal(n)))
    h = dict(x=bf16(2 * g.standard_normal((M, C))), y=bf16(g.standard_normal((M, C))),
             mod=bf16(0.3 * g.standard_normal((2, 4 * C))), pos=g.integers(0, 40, (M // 2, 3)).astype(np.int32),
             qn=bf16(1 + 0.1 * g.standard_normal(128)), kn=bf16(1 + 0.1 * g.standard_normal(128)))
    d = {k: (dev(v) if k == "pos" else dev_bf16(v)) for k, v in h.items()}
    dw = {k: (dev(v[0]), dev(v[1]), dev(v[2]), dev_bf16(v[3])) for k, v in w.items()}
    return h, w, d, dw


def _run(d, dw, stream=None):
    import bit_diffusion_transformer_svdq_amd as P
    m = d["mod"]
    gate, scale, shift, gate2 = (m[:, i * C:(i + 1) * C] for i in range(4))
    kw = dict(stream=stream)
    h, (q8, s8) = P.gate_norm_modulate(d["x"], d["y"], gate=gate, scale=scale, shift=shift, quantize="int8",
                                       smooth=dw["qkv"][0], **kw)
    qkv = P.w8a8_gemm(q8, s8, *dw["qkv"][1:], **kw)
    E = HEADS * 128
    q, k = P.rope_axes(qkv[:, :E].unflatten(1, (HEADS, 128)), qkv[:, E:2 * E].unflatten(1, (HEADS, 128)), d["pos"], AXES,
                       q_norm=d["qn"], k_norm=d["kn"], **kw)
    _, (q8, s8) = P.gate_norm_modulate(h, scale=scale, shift=shift, quantize="int8", smooth=dw["up"][0], **kw)
    u = P.w8a8_gemm(q8, s8, *dw["up"][1:], epilogue="gelu_tanh", **kw)
    q8, s8 = P.quantize_act_int8(u, dw["down"][0], **kw)
    v = P.w8a8_gemm(q8, s8, *dw["down"][1:], **kw)
    h2, z = P.gate_norm_modulate(h, v, post_norm="rms", gate=gate2, norm="rms", **kw)
    return h, qkv, q, k, u, v, h2, z


def _relative(a, b):
    return np.linalg.norm(host(a) - b) / np.linalg.norm(b)


def test_block_against_the_oracle(block):
    """Stage by stage from the device's own inputs; the int8 stages differ from the
    oracle's by code steps at rounding borders only, so their relative error
    stays near the bf16 rounding (2^-8 / sqrt 3 on average)."""
    h, w, d, dw = block
    got = _run(d, dw)
    m = h["mod"]
    gate, scale, shift, gate2 = (m[:, i * C:(i + 1) * C] for i in range(4))
    h1, z1 = B.gate_norm_modulate(h["x"], h["y"], gate=gate, scale=scale, shift=shift)
    assert _relative(got[0], h1) < 2.0 ** -8

    def linear(z, name, epi="none"):
        sm, wc, ws, b = w[name]
        v = z / sm.astype(np.float64)
        s, inv = B.token_scales(v)
        return B.w8a8_gemm(np.rint(v * inv[:, None]).astype(np.int8), s, wc, ws, b, epi)[0]

    assert _relative(got[1], linear(z1, "qkv")) < 2.0 ** -8
    E = HEADS * 128
    for i, n in ((0, "qn"), (1, "kn")):
        t = host(got[1])[:, i * E:(i + 1) * E].reshape(M, HEADS, 128)
        assert _relative(got[2 + i], B.rope_axes(t, h["pos"], AXES, norm_weight=h[n])) < 2.0 ** -8
    _, z2 = B.gate_norm_modulate(host(got[0]), scale=scale, shift=shift)
    assert _relative(got[4], linear(z2, "up", "gelu_tanh")) < 2.0 ** -7
    qd, sd = B.quantize_act_int8(host(got[4]), w["down"][0])
    assert _relative(got[5], B.w8a8_gemm(qd, sd, *w["down"][1:])[0]) < 2.0 ** -8
    h3, z3 = B.gate_norm_modulate(host(got[0]), host(got[5]), post_norm="rms", gate=gate2, norm="rms")
    assert _relative(got[6], h3) < 2.0 ** -8 and _relative(got[7], z3) < 2.0 ** -8


def test_graph_replays(block):
    """Two captured graphs replayed in turn, with eager work on the same stream in
    between: every output bit for bit the eager one."""
    import torch
    _, _, d, dw = block
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        want = [t.clone() for t in _run(d, dw)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = _run(d, dw)
        graphs.append((g, out))
    for rep in range(3):
        with torch.cuda.stream(s):
            for g, out in graphs:
                for t in out:
                    t.fill_(7)
                g.replay()
                again = _run(d, dw)
        torch.cuda.synchronize()
        for out in (graphs[0][1], graphs[1][1], again):
            for t, w in zip(out, want):
                assert torch.equal(t, w), rep


def test_another_stream(block):
    """The calls on a stream given by hand, ordered by the caller."""
    import torch
    _, _, d, dw = block
    want = [t.clone() for t in _run(d, dw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(d, dw, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for t, w in zip(got, want):
        assert torch.equal(t, w)


def test_few_tokens_give_the_rows_of_many(block):
    """Row r of the 8-bit product does not depend on how many rows run with it
    (integer sums): the few-token kernel and the tiles agree bit for bit."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    _, _, d, dw = block
    q, s = P.quantize_act_int8(d["x"], dw["up"][0])
    full = P.w8a8_gemm(q, s, *dw["up"][1:])
    for m in (1, 2, 16, 17, 33, 64, 65, 100):
        assert torch.equal(P.w8a8_gemm(q[:m].contiguous(), s[:m].contiguous(), *dw["up"][1:]), full[:m]), m
