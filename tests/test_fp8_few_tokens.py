"""Up to 16 tokens of the 8-bit floating-point products where K is long: which of the two
kernels takes them (seen in the workspace that a call asks for), and their values.  Bounds:
tests/fp8_util.py."""
import numpy as np
import pytest
import torch  # noqa: F401  (ahead of the library, so that both use one HIP runtime)

import oracle.fp8_oracle as F
from bit_diffusion_transformer_svdq_amd._lib import lib
from tests.block_util import bf16, check, dev, dev_bf16, host
from tests.fp8_util import dev_codes, product_bound, tokens, weights
from tests.test_fp8_gated_gpu import _check_out

COUNTERS = 1 << 20


def _need(M, N, K, form):
    L = lib()
    return L.svdq_fp8_gemm_workspace_size(M, N, K) if form == "plain" else \
        L.svdq_fp8_gated_gemm_workspace_size(M, N, K, int(form == "codes"))


@pytest.mark.parametrize("M", [1, 4])
@pytest.mark.parametrize("form,N,K", [("plain", 64, 65536), ("plain", 1024, 16384), ("plain", 2048, 32768), ("gated", 1024, 8192),
                                      ("codes", 64, 65536), ("codes", 2048, 32768)])
def test_long_k_is_divided(form, N, K, M):
    """N / 16 workgroups of the few-token kernel would leave most of the chip idle: the
    tiles split K (partials in the workspace, more than the few-token kernel's codes take)."""
    assert _need(M, N, K, form) > COUNTERS + 64 * N


@pytest.mark.parametrize("form,N,K,M", [("plain", 64, 8192, 4), ("plain", 4096, 65536, 1), ("gated", 4096, 8192, 4), ("gated", 64, 4096, 16)])
def test_the_weight_stream_needs_no_workspace(form, N, K, M):
    assert _need(M, N, K, form) == 0


def test_codes_of_the_weight_stream():
    for M, K in ((1, 16384), (4, 16384), (16, 8192)):
        assert _need(M, 320, K, "codes") == COUNTERS + 320 * 64


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 4, 5, 16])
@pytest.mark.parametrize("N,K", [(64, 65536), (192, 16448), (4160, 16384), (320, 8256), (4096, 4160)])
@pytest.mark.parametrize("form", ["plain", "gated", "codes"])
def test_values(M, N, K, form):
    import bit_diffusion_transformer_svdq_amd as P
    x, w = tokens(M, K, 13), weights(N, K, 13)
    g = np.random.default_rng([M, N, K])
    b = bf16(0.3 * g.standard_normal(N))
    if form == "plain":
        y = host(P.fp8_gemm(dev_codes(x[0]), dev(x[1]), dev_codes(w[0]), dev(w[1]), dev_bf16(b)))
        v, mags = F.product(*x, *w, b)
        check(y, v, product_bound(K, mags, v))
        return
    x, up = (x[0], x[1] * np.float32(0.1)), weights(N, K, 113)
    got = P.fp8_gated_gemm(dev_codes(x[0]), dev(x[1]), dev_codes(w[0]), dev(w[1]), dev_codes(up[0]), dev(up[1]), dev_bf16(b),
                           quantize="fp8" if form == "codes" else None)
    _check_out(got, x, w, up, (b, None), "silu")
