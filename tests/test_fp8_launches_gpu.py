"""Products of the 8-bit floating-point linear that run as two launches, whole rounds of a
large tile and the rest on another.  Each case is captured, and its graph must hold two
kernels, so that no case can pass on one launch.  Needs an MI355X.  Bounds:
tests/fp8_util.py."""
import ctypes

import numpy as np
import pytest

from tests.block_util import bf16, check, dev, dev_bf16, host
from tests.fp8_util import dev_codes, product_bound, tokens, weights
from tests.test_fp8_gated_gpu import _check_out

import oracle.fp8_oracle as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_diffusion_transformer_svdq_amd import check_device
    check_device(0)


def _kernels(call):
    """The number of kernels of a captured call that allocates nothing, and that of its
    other nodes."""
    import torch
    from bit_diffusion_transformer_svdq_amd._lib import lib
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    L, graph, n = lib(), ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert L.hipGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert L.hipGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    kinds = []
    for node in nodes[:n.value]:
        kind = ctypes.c_int(-1)
        assert L.hipGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kinds.append(kind.value)
    return kinds.count(0), len(kinds) - kinds.count(0)   # hipGraphNodeTypeKernel is 0


def _inside(s, before, behind):
    """Scales as a part of a larger array, whose rest are NaN."""
    import torch
    whole = torch.full((s.shape[0], before + s.shape[1] + behind), float("nan"), device="cuda")
    whole[:, before:before + s.shape[1]] = dev(s)
    return whole[:, before:before + s.shape[1]]


def _some(M):
    """Tokens from everywhere, the last 150 and those around the ends of tiles."""
    ends = np.concatenate([np.arange(0, M, 256) + i for i in (-1, 0, 1)])
    rows = np.unique(np.concatenate([np.arange(0, M, 61), np.arange(M - 150, M), ends]))
    return rows[(rows >= 0) & (rows < M)]


# the rest on one tile after the other of the smaller ones, and split over K
@pytest.mark.parametrize("M,N,K,splits", [(4112, 6144, 512, False), (4112, 4096, 960, False), (2200, 8192, 960, False),
                                          (4160, 4096, 2112, True), (2064, 8192, 2112, True)])
def test_gemm(M, N, K, splits):
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd._lib import lib
    x, w = tokens(M, K, 11), weights(N, K, 11)
    b = bf16(np.random.default_rng(N).standard_normal(N))
    need = lib().svdq_fp8_gemm_workspace_size(M, N, K)
    assert (need > 0) == splits    # the first launch is never split
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    behind = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = behind[:M]
    a = dev_codes(x[0]), _inside(x[1], 3, 6), dev_codes(w[0]), dev(w[1]), dev_bf16(b)

    def call():
        P.fp8_gemm(*a, out=y, workspace=ws)
    call()
    first = y.clone()
    assert _kernels(call) == (2, 0)
    for _ in range(3):
        y.fill_(7)
        call()
        assert torch.equal(y, first)
    assert bool((behind[M:] == 7).all())
    if splits:
        assert not bool(ws[:1 << 20].any())
    else:
        P.debug_set_fp8_plan(442, 1)
        try:
            one = P.fp8_gemm(*a)
        finally:
            P.debug_set_fp8_plan()
        assert torch.equal(first, one)
    rows = _some(M)
    v, mags = F.product(x[0][rows], x[1][:, rows], *w, b)
    check(host(first[torch.from_numpy(rows).cuda()]), v, product_bound(K, mags, v))


@pytest.mark.parametrize("M,N,K,quantize,splits", [
    (2200, 4096, 960, None, False), (4112, 6144, 512, None, False), (2064, 4096, 2112, None, True),
    (2200, 6144, 512, "fp8", False), (4112, 6144, 512, "fp8", False), (2064, 4096, 2112, "fp8", True),
    (4160, 2048, 2112, "fp8", True)])
def test_gated(M, N, K, quantize, splits):
    import torch
    import bit_diffusion_transformer_svdq_amd as P
    from bit_diffusion_transformer_svdq_amd._lib import lib
    x, gate, up = tokens(M, K, 12), weights(N, K, 12), weights(N, K, 112)
    x = x[0], x[1] * np.float32(0.2)
    g = np.random.default_rng([M, N, K])
    b = [bf16(0.3 * g.standard_normal(N)) for _ in range(2)]
    sm = np.exp(0.7 * g.standard_normal(N)).astype(np.float32) if quantize else None
    need = lib().svdq_fp8_gated_gemm_workspace_size(M, N, K, int(quantize is not None))
    assert (need > 0) == splits
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    a = [dev_codes(x[0]), _inside(x[1], 1, 4), dev_codes(gate[0]), dev(gate[1]), dev_codes(up[0]), dev(up[1]), *map(dev_bf16, b)]
    kw = dict(quantize=quantize, smooth=None if sm is None else dev(sm))
    if quantize:
        whole = torch.full((N // 128, M + 7), -3.0, device="cuda")
        codes = torch.full((M + 3, N), 7, dtype=torch.uint8, device="cuda")
        out = codes[:M].view(torch.float8_e4m3fn), whole[:, 2:M + 2]
        parts = [codes[:M], out[1]]
    else:
        out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
        parts = [out]

    def call():
        P.fp8_gated_gemm(*a, **kw, out=out, workspace=ws)
    call()
    first = [t.clone() for t in parts]
    assert _kernels(call) == (2, 0)
    for _ in range(3):
        for t in parts:
            t.fill_(7)
        call()
        assert all(torch.equal(t, f) for t, f in zip(parts, first))
    if quantize:
        assert bool((whole[:, :2] == -3).all()) and bool((whole[:, M + 2:] == -3).all()) and bool((codes[M:] == 7).all())
    if splits:
        assert not bool(ws[:1 << 20].any())
    else:
        P.debug_set_fp8_plan(442, 1)
        try:
            one = P.fp8_gated_gemm(*a, **kw)
        finally:
            P.debug_set_fp8_plan()
        one = [one[0].view(torch.uint8), one[1]] if quantize else [one]
        assert all(torch.equal(t, f) for t, f in zip(one, first))
    rows = _some(M)
    at = torch.from_numpy(rows).cuda()
    got = (first[0][at].view(torch.float8_e4m3fn), first[1][:, at]) if quantize else first[0][at]
    _check_out(got, (x[0][rows], x[1][:, rows]), gate, up, b, "silu", sm)
