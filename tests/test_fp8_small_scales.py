"""Scales at the lower end of fp32.  In a last block of 64 channels the kernels add the
products twice and halve the weights' scale, which counts as the even multiple of 2^-149
next to it there (include/svdq.h).  Needs an MI355X."""
import numpy as np
import pytest
import torch  # noqa: F401  (ahead of the library, so that both use one HIP runtime)

import oracle.fp8_oracle as F
from tests.block_util import bf16, dev, host
from tests.fp8_util import dev_codes

pytestmark = pytest.mark.gpu
SMALL = F.encode(np.arange(-4, 5).astype(float))


@pytest.mark.parametrize("M,tile", [(1, 0), (16, 0), (16, 1), (70, 0), (300, 0), *[(130, t) for t in (114, 213, 224, 413, 423, 432, 442)]])
@pytest.mark.parametrize("K", [64, 192, 576])
@pytest.mark.parametrize("side", ["weights", "tokens"])
def test_subnormal_scales(M, tile, K, side):
    """Whole numbers and scales of 2^-149 (a token's) or 3 2^-148 (the weights') and 2^127:
    every sum is exact."""
    import bit_diffusion_transformer_svdq_amd as P
    N, KB = 192, -(-K // 128)
    g = np.random.default_rng([M, K, side == "weights"])
    tiny, big = np.float32(2.0 ** -149 if side == "tokens" else 3 * 2.0 ** -148), np.float32(2.0 ** 127)
    sx = np.full((KB, M), tiny if side == "tokens" else big, np.float32)
    sw = np.full((2, KB), tiny if side == "weights" else big, np.float32)
    x = SMALL[g.integers(0, 9, (M, K))], sx
    w = SMALL[g.integers(0, 9, (N, K))], sw
    want = F.product(*x, *w)[0]
    assert np.abs(want).max() > 0
    P.debug_set_fp8_plan(tile, 0)
    try:
        y = P.fp8_gemm(dev_codes(x[0]), dev(sx), dev_codes(w[0]), dev(sw))
        gate = np.zeros((N, K), np.uint8)
        gate[:, -1] = F.encode(64.0)
        x[0][:, -1] = F.encode(256.0)
        h = P.fp8_gated_gemm(dev_codes(x[0]), dev(sx), dev_codes(gate), dev(sw), dev_codes(w[0]), dev(sw))
    finally:
        P.debug_set_fp8_plan()
    assert np.array_equal(host(y), bf16(want))
    gv, u = F.product(*x, gate, sw)[0], F.product(*x, *w)[0]
    assert (gv == (2.0 ** -8 if side == "tokens" else 6 * 2.0 ** -8)).all()   # 64 * 256 * tiny * big
    ref = F.silu(gv) * u
    assert (np.abs(host(h) - ref) <= (2.0 ** -8 + 16 * 2.0 ** -24) * np.abs(ref)).all()


@pytest.mark.parametrize("M", [3, 70, 300])
def test_odd_multiples_in_half_a_block(M):
    """As stated: 5 2^-149 of the weights counts as 4 2^-149 (ties to even) in the block of 64, as
    itself in the whole one before it."""
    import bit_diffusion_transformer_svdq_amd as P
    N, K = 64, 192
    g = np.random.default_rng(M)
    x = SMALL[g.integers(0, 9, (M, K))], np.full((2, M), 2.0 ** 127, np.float32)
    w = SMALL[g.integers(0, 9, (N, K))], np.full((1, 2), 5 * 2.0 ** -149, np.float32)
    y = P.fp8_gemm(dev_codes(x[0]), dev(x[1]), dev_codes(w[0]), dev(w[1]))
    w[1][0, 1] = 4 * 2.0 ** -149
    assert np.array_equal(host(y), bf16(F.product(*x, *w)[0]))
