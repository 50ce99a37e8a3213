"""Outputs of the 8-bit floating-point operators that lie beyond 4 GiB of their array's
start.  Needs an MI355X.  Bounds: tests/fp8_util.py."""
import numpy as np
import pytest

import oracle.fp8_oracle as F
from tests.block_util import dev, gate_norm_bound, host
from tests.fp8_util import dev_codes, host_codes, tokens, weights
from tests.test_fp8_gated_gpu import _check_out, check_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)
    yield
    torch.cuda.empty_cache()


def _rows(M, border):
    return np.r_[0:8, border - 8:border + 8, M - 40:M]


@pytest.mark.parametrize("M,quantize", [(40000, None), (70000, "fp8")])
def test_gated(M, quantize):
    """bf16 rows and codes, the codes' scales in rows of an array of 8 GiB."""
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    N, K = 65536, 64
    x, gate, up = tokens(M, K, 1), weights(N, K, 1), weights(N, K, 101)
    out = None
    if quantize:
        whole = torch.full((N // 128, 4 << 20), 7.0, device="cuda")
        out = torch.empty((M, N), dtype=torch.float8_e4m3fn, device="cuda"), whole[:, -M - 3:-3]
    got = P.fp8_gated_gemm(dev_codes(x[0]), dev(x[1]), dev_codes(gate[0]), dev(gate[1]), dev_codes(up[0]), dev(up[1]),
                           quantize=quantize, out=out)
    rows = _rows(M, 65536 if quantize else 32768)   # the 4 GiB border
    at = torch.from_numpy(rows).cuda()
    part = (torch.stack([got[0].view(torch.uint8)[r] for r in rows]).view(torch.float8_e4m3fn), got[1][:, at]) if quantize else \
        torch.stack([got[r] for r in rows])
    _check_out(part, (x[0][rows], x[1][:, rows]), gate, up, (None, None), "silu")
    if quantize:
        assert bool((whole[:, -3:] == 7).all()) and bool((whole[:, :-M - 3] == 7).all())


def test_quantizer():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    M, K = 70000, 65536
    x = torch.randn((M, K), dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    q, s = P.quantize_act_fp8(x)
    for r in np.split(_rows(M, 65536), 4):
        want = F.quantize_act_fp8(np.stack([host(x[i]) for i in r]))
        assert np.array_equal(np.stack([host_codes(q[i]) for i in r]), want[0])
        assert np.array_equal(np.stack([s[:, i].cpu().numpy() for i in r], 1), want[1])


def test_norm():
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    M, C = 140000, 32768
    x = torch.randn((M, C), dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    _, (q, s) = P.gate_norm_modulate(x, norm="rms", quantize="fp8")
    for r in np.split(_rows(M, 131072), 4):
        _, _, z, ez = gate_norm_bound(np.stack([host(x[i]) for i in r]), norm="rms")
        check_codes(np.stack([host_codes(q[i]) for i in r]), np.stack([s[:, i].cpu().numpy() for i in r], 1), z, ez)
