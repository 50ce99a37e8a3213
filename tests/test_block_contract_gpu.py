"""What the block operators' contract says, on a device.  Needs an MI355X."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


@pytest.mark.parametrize("M,C", [(1, 64), (3, 72), (5, 1536), (2, 8200), (2100, 320)])
@pytest.mark.parametrize("parts", ["y", "gate", "y and gate"])
def test_a_stream_that_is_its_own_block_output_or_gate(M, C, parts):
    """The stream updated in place where y, or a gate of M rows, is the stream too:
    what the call gives out of place; what is not in place is refused."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    g = torch.Generator().manual_seed(C)
    x, y, gate = (torch.randn(M, C, generator=g).cuda().bfloat16() for _ in range(3))
    mod = torch.randn(1, 2 * C, generator=g).cuda().bfloat16()
    kw = dict(scale=mod[:, :C], shift=mod[:, C:], norm="rms")
    y = x if "y" in parts.split(" and ") else y
    gate = x if "gate" in parts.split(" and ") else gate
    h0, z0 = (t.clone() for t in P.gate_norm_modulate(x, y, gate=gate, **kw))
    for key in ("scale", "shift"):   # read after h is written
        with pytest.raises(P.SvdqError):
            P.gate_norm_modulate(x, y, gate=gate, norm="rms", h_out=x, **{key: x})
    h, z = P.gate_norm_modulate(x, y, gate=gate, h_out=x, **kw)
    assert h is x and torch.equal(x, h0) and torch.equal(z, z0)
    assert bool(np.isfinite(x.float().cpu().numpy()).all())


def _angle_bound(pos, axes, theta, spectrum):
    """Error of an angle, kernel and oracle together, in radians: both keep a rate to 64 bits
    (the kernel's, step j of a running product, to 1.5 j + 2 ln(1/rate) + 2 of them, the oracle's
    exponential to ln(1/rate) + 4), products and reductions below 2^-44."""
    n = [d // 2 for d in axes]
    j = np.concatenate([np.arange(k) for k in n]) if spectrum == "axis" else np.arange(sum(n))
    per = np.repeat(n, n) if spectrum == "axis" else np.full(sum(n), sum(n))
    fall = j / per * np.log(theta)   # ln(1 / rate)
    own = np.repeat(np.arange(len(axes)), n)
    return 2.0 ** -44 + np.abs(pos[:, own].astype(np.float64)) * np.exp(-fall) * (1.5 * j + 3 * fall + 6) * 2.0 ** -63


@pytest.mark.parametrize("axes", [(128,), (16, 56, 56), (2,), (64, 64, 64, 64)])
@pytest.mark.parametrize("spectrum", ["axis", "shared"])
@pytest.mark.parametrize("theta", [1e4, 1e6])
@pytest.mark.parametrize("kind", ["int", "float"])
def test_far_positions_keep_the_precision_of_near_ones(axes, spectrum, theta, kind):
    """Up to 2^31 the tables are rounded once: half a step below one, 2^-25, beyond the
    angle's own error."""
    import oracle.block_oracle as B
    import bit_diffusion_transformer_svdq_amd as P
    from tests.block_util import dev, host
    g = np.random.default_rng([3, len(axes)])
    pos = g.integers(-2 ** 31, 2 ** 31 - 1, (600, len(axes)))
    pos[0], pos[1] = -2 ** 31, 2 ** 31 - 1
    pos = pos.astype(np.int32 if kind == "int" else np.float32)
    t = B.rope_angles(pos, axes, theta, spectrum)
    e = 2.0 ** -25 + _angle_bound(pos, axes, theta, spectrum)
    c, s = P.rope_axes_tables(dev(pos), axes, theta=theta, spectrum=spectrum)
    assert (np.abs(host(c) - np.cos(t)) <= e).all() and (np.abs(host(s) - np.sin(t)) <= e).all()


def test_positions_too_far_for_an_angle_still_turn():
    """fp32 positions up to the largest: whatever the angle, a cosine and a sine of one."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from tests.block_util import dev, host
    pos = np.array([[s * 2.0 ** k] for k in range(32, 128) for s in (1.0, -1.9999999)], np.float32)
    assert np.isfinite(pos).all()
    c, s = (host(t) for t in P.rope_axes_tables(dev(pos), (64,)))
    # two values rounded to fp32 on the circle: |c dc| + |s ds| <= 2^-25 (|c| + |s|), twice
    assert (np.abs(c * c + s * s - 1) <= 2 * 2.0 ** -25 * np.sqrt(2) + 2.0 ** -40).all()
    q = torch.randn(len(pos), 2, 64, device="cuda").bfloat16()
    qo, _ = P.rope_axes(q, None, dev(pos), (64,))
    n0, n1 = (t.float().view(-1, 2, 32, 2).square().sum(-1) for t in (q, qo))
    assert bool(((n0 - n1).abs() <= 2.0 ** -6 * n0).all())


@pytest.mark.parametrize("M", [2, 300])
def test_gelu_to_the_end_of_its_tail(M):
    """Exact arguments from -12 to -8.  While 2^t = exp(-2u) stays below 2^126 the relative
    error is the function's own, (3.5 t + 7) 2^-24, and the rounding to bf16; beyond, where the
    value is below 10.1 2^-126, it may come out as zero."""
    import bit_diffusion_transformer_svdq_amd as P
    from tests.block_util import U, dev, dev_bf16, host
    qx, qw = np.zeros((M, 64), np.int8), np.zeros((256, 64), np.int8)
    qx[:, 5] = 1
    qw[:, 5] = np.arange(-128, 128)
    b = np.full(256, -10.0)
    y = host(P.w8a8_gemm(dev(qx), dev(np.full(M, 2.0 ** -6, np.float32)), dev(qw), dev(np.ones(256, np.float32)), dev_bf16(b),
                         epilogue="gelu_tanh"))
    x = b + np.arange(-128, 128) / 64.0
    u = np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    t = -2 * u * np.log2(np.e)
    want = x / (1 + np.exp(-2 * u))
    near = t < 125.9
    rel = 2.0 ** -8 / (1 + 2.0 ** -8) + 1.01 * (3.5 * t + 7) * U
    assert near.sum() > 100 and (~near).sum() > 100
    assert (np.abs(y - want) <= rel * np.abs(want))[:, near].all()
    assert (np.abs(want[~near]) <= 10.1 * 2.0 ** -125.9).all()
    assert ((y[:, ~near] <= 0) & (y[:, ~near] >= (1 + rel[~near]) * want[~near])).all()


def test_outputs_given_with_another_stream_outlive_their_owner():
    """An output given with a stream and freed at once is not handed out again while
    that stream still has it to write; the stream is busy throughout."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    x = torch.randn(64, 4096, device="cuda").bfloat16()
    want = P.quantize_act_int8(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = (torch.empty(64, 4096, dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda"))
    at = out[0].data_ptr()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    P.quantize_act_int8(x, out=out, stream=s)
    del out
    more = [torch.empty(64, 4096, dtype=torch.int8, device="cuda") for _ in range(4)]
    assert not s.query(), "the stream ended before the memory was asked for"
    assert all(t.data_ptr() != at for t in more)
    for t in more:
        t.fill_(7)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in more)
    assert torch.equal(P.quantize_act_int8(x)[0], want[0])


def test_one_row_through_the_library_with_strides_of_nothing():
    """M = 1: the strides of x, y and h are not read."""
    import ctypes
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd._lib import SUCCESS, lib
    C = 320
    x, y, h = (torch.randn(1, C, device="cuda").bfloat16() for _ in range(3))
    z = torch.empty(1, C, device="cuda", dtype=torch.bfloat16)
    want = P.gate_norm_modulate(x, y, norm="rms")
    p = [ctypes.c_void_p(t.data_ptr()) for t in (x, y, h, z)]
    st = lib().svdq_gate_norm_modulate(p[0], 0, 0, p[1], -8, 0, None, None, 0, 0, 1.0, 2, None, None, None, 0, 0, 1e-6, 1, C,
                                       p[2], 3, 0, None, p[3], None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == SUCCESS
    assert torch.equal(h, want[0]) and torch.equal(z, want[1])
