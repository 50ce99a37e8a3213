"""Random shapes of the 8-bit floating-point products on the plans that the sizes choose,
with token scales and codes that are parts of larger arrays.  Needs an MI355X.  Bounds:
tests/fp8_util.py."""
import numpy as np
import pytest

import oracle.fp8_oracle as F
from tests.block_util import bf16, check, dev, dev_bf16, host
from tests.fp8_util import act_bound, dev_codes, product_bound, tokens, weights
from tests.test_fp8_gated_gpu import _check_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _part(c, s, g):
    """The tokens' codes and scales inside of larger arrays: codes from a row on, scales from
    any token on and rows apart."""
    import torch
    M, before, behind = c.shape[0], int(g.integers(0, 4)), int(g.integers(0, 6))
    codes = torch.full((before + M + behind, c.shape[1]), 0x7f, dtype=torch.uint8, device="cuda")
    scales = torch.full((s.shape[0], before + M + behind), float("nan"), device="cuda")
    codes[before:before + M], scales[:, before:before + M] = dev(c), dev(s)
    return codes.view(torch.float8_e4m3fn)[before:before + M], scales[:, before:before + M]


def _sizes(g):
    M = int(np.exp(g.uniform(0, np.log(1500))))
    N, K = (64 * int(np.exp(g.uniform(0, np.log(48)))) for _ in range(2))
    return M, N, K


@pytest.mark.parametrize("seed", range(24))
def test_gemm(seed):
    import bit_diffusion_transformer_svdq_amd as P
    g = np.random.default_rng([seed, 7])
    M, N, K = _sizes(g)
    print("gemm", seed, M, N, K, flush=True)
    x, w = tokens(M, K, seed), weights(N, K, seed)
    x = x[0], x[1] * np.float32(0.2)
    b = bf16(g.standard_normal(N)) if g.integers(2) else None
    epilogue = ["none", "gelu_tanh"][g.integers(2)]
    y = P.fp8_gemm(*_part(*x, g), dev_codes(w[0]), dev(w[1]), dev_bf16(b), epilogue=epilogue)
    v, mags = F.product(*x, *w, b)
    err = product_bound(K, mags, v)
    if epilogue == "gelu_tanh":
        err, v = act_bound(v, err), F.gelu_tanh(v)
    check(host(y), v, err)


@pytest.mark.parametrize("seed", range(24))
def test_gated(seed):
    import torch

    import bit_diffusion_transformer_svdq_amd as P
    g = np.random.default_rng([seed, 8])
    M, N, K = _sizes(g)
    print("gated", seed, M, N, K, flush=True)
    x, gate, up = tokens(M, K, seed), weights(N, K, seed), weights(N, K, seed + 100)
    x = x[0], x[1] * np.float32(0.2)
    b = [bf16(0.3 * g.standard_normal(N)) if g.integers(2) else None for _ in range(2)]
    act, coded = ["silu", "gelu_tanh"][g.integers(2)], bool(g.integers(2))
    sm = np.exp(0.7 * g.standard_normal(N)).astype(np.float32) if coded and g.integers(2) else None
    out = None
    if coded:  # scales into a part of a larger array, whose rest stays
        whole = torch.full((-(-N // 128), M + 5), -3.0, device="cuda")
        out = torch.empty(M, N, dtype=torch.float8_e4m3fn, device="cuda"), whole[:, 2:M + 2]
    got = P.fp8_gated_gemm(*_part(*x, g), dev_codes(gate[0]), dev(gate[1]), dev_codes(up[0]), dev(up[1]), dev_bf16(b[0]),
                           dev_bf16(b[1]), activation=act, quantize="fp8" if coded else None,
                           smooth=None if sm is None else dev(sm), out=out)
    _check_out(got, x, gate, up, b, act, sm)
    if coded:
        assert (whole[:, :2] == -3).all() and (whole[:, M + 2:] == -3).all()
