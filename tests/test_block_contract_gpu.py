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
