"""What is measured of the 8-bit floating-point linear (e4m3 codes, one scale per token
and 128 channels of K, one per 128 x 128 weights), the gated feed-forward block on it
(both projections, the activation and the product in one kernel) and the norms that
write such codes.

``run`` computes a case in its plain form (elementary torch operations in 32 bits)
or, where ``own`` is true, with the package's operators.  Sizes follow a 12B-class
diffusion transformer at 1024² (hidden 3072, 4096 image and 512 text tokens, MLP
12288) and generic smaller and odd ones.
"""
from __future__ import annotations

import math

import torch

own = False

GELU_C = math.sqrt(2.0 / math.pi)
BLOCK = 128       # channels of K that share a scale; rows and columns of the weights that do
LARGEST = 448.0   # of e4m3


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one conditioning vector through an embedder's second linear: latency
        dict(name="linear 1 token", op="linear", M=1, K=3072, N=3072, smooth=False, bias=True, epilogue="none"),
        # a text prompt into the model's width
        dict(name="linear 77 tokens", op="linear", M=77, K=4096, N=1536, smooth=False, bias=True, epilogue="none"),
        # a patch sequence of an odd picture, half a scale block at the end of N
        dict(name="linear 1333 tokens", op="linear", M=1333, K=1920, N=7744, smooth=True, bias=True,
             epilogue="gelu_tanh"),
        # the MLP up-projection of all 4608 tokens of a 1024² image
        dict(name="linear 4608 tokens", op="linear", M=4608, K=3072, N=12288, smooth=True, bias=True,
             epilogue="gelu_tanh"),
        # the gated embedder of a pooled vector: latency
        dict(name="gated 1 token", op="gated", M=1, K=2304, F=6144, smooth=False, bias=False, act="silu"),
        # both projections of a short text stream, half a scale block at the end of K and F
        dict(name="gated 300 tokens", op="gated", M=300, K=1856, F=5056, smooth=True, bias=True, act="gelu_tanh"),
        # of one odd picture
        dict(name="gated 4173 tokens", op="gated", M=4173, K=2304, F=6144, smooth=True, bias=False, act="silu"),
        # the whole feed-forward block of a few tokens (learned queries of an adapter)
        dict(name="ffn 16 tokens", op="ffn", M=16, C=1536, F=4096, smooth=False, bias=False, act="silu"),
        # of the text stream
        dict(name="ffn 512 tokens", op="ffn", M=512, C=3840, F=10240, smooth=True, bias=True, act="silu"),
        # of all tokens of a 1024² image
        dict(name="ffn 4608 tokens", op="ffn", M=4608, C=3072, F=8192, smooth=True, bias=False, act="silu"),
        # gated residual and norm into codes, and the up-projection of 64 tokens
        dict(name="norm + linear 64", op="norm_linear", M=64, B=1, C=3072, N=12288, norm="layer",
             epilogue="gelu_tanh"),
        # two pictures' norm into codes and their fused QKV projection
        dict(name="norm + linear 2 x 2045", op="norm_linear", M=4090, B=2, C=2304, N=6912, norm="rms",
             epilogue="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "ffn", "ffn", "norm_linear"])
    K, N, M = 64 * _log(rng, 4, 192), 64 * _log(rng, 2, 192), _log(rng, 1, 4608)
    smooth, bias = rng.random() < 0.5, rng.random() < 0.5
    if op == "linear":
        M = max(1, min(M, 4608 * 3072 * 12288 // (K * N)))
        return dict(op=op, M=M, K=K, N=N, smooth=smooth, bias=bias, epilogue=rng.choice(["none", "gelu_tanh"]))
    act = rng.choice(["silu", "silu", "gelu_tanh"])
    if op == "gated":
        M = max(1, min(M, 4608 * 3072 * 12288 // (2 * K * N)))
        return dict(op=op, M=M, K=K, F=N, smooth=smooth, bias=bias, act=act)
    C = 64 * _log(rng, 4, 64)
    if op == "ffn":
        M = max(1, min(M, 4608 * 3072 * 8192 // (C * N)))
        return dict(op=op, M=M, C=C, F=N, smooth=smooth, bias=bias, act=act)
    B = rng.choice([1, 1, 2, 3])
    S = max(1, min(M, 4608 * 3072 * 12288 // (C * N)) // B)
    return dict(op=op, M=B * S, B=B, C=C, N=N, norm=rng.choice(["layer", "rms"]),
                epilogue=rng.choice(["none", "gelu_tanh"]))


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activations(g, M, C):
    """Unit normal rows with 1 % of the channels 30 times as large."""
    x = _normal(g, M, C)
    loud = torch.randperm(C, generator=g, device="cuda")[:max(1, C // 100)]
    x[:, loud] *= 30.0
    return x


def _smoothing(x):
    """A layer's smoothing vector: larger where its activations are."""
    return (x.float().abs().amax(0).clamp(min=1e-2) / 0.08).sqrt()


def _weights(g, N, K, smooth):
    """e4m3 codes and 128 x 128 block scales of N(0, 0.02) weights, smoothing moved into them."""
    w = _normal(g, N, K, std=0.02)
    if smooth is not None:
        w = w * smooth
    n, k = -(-N // BLOCK), -(-K // BLOCK)
    whole = torch.zeros(n * BLOCK, k * BLOCK, device="cuda")
    whole[:N, :K] = w
    s = (whole.view(n, BLOCK, k, BLOCK).abs().amax((1, 3)) / LARGEST).contiguous()
    wide = s.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:N, :K]
    return (w / wide).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, st, bf = case["op"], dict(case), torch.bfloat16
    M = case["M"]
    if op == "norm_linear":
        B, C, N = case["B"], case["C"], case["N"]
        st["x"] = _activations(g, M, C).to(bf)
        st["y"] = _normal(g, M, C, std=0.7).to(bf)
        # one projection gives every vector of the block: strided chunks of it
        mod = _normal(g, B, 3 * C, std=0.3).to(bf)
        st["gate"], st["scale"], st["shift"] = mod[:, :C], mod[:, C:2 * C], mod[:, 2 * C:]
        st["sm"] = torch.exp(_normal(g, C, std=0.3))
        st["w"] = _weights(g, N, C, st["sm"])
        st["b"] = _normal(g, N, std=0.01).to(bf)
        return st
    K = case["C"] if op == "ffn" else case["K"]
    st["x"] = _activations(g, M, K).to(bf)
    st["sm"] = _smoothing(st["x"]) if case["smooth"] else None
    if op == "linear":
        st["w"] = _weights(g, case["N"], K, st["sm"])
        st["b"] = _normal(g, case["N"], std=0.01).to(bf) if case["bias"] else None
        return st
    F = case["F"]
    st["w_gate"], st["w_up"] = _weights(g, F, K, st["sm"]), _weights(g, F, K, st["sm"])
    st["b_gate"] = _normal(g, F, std=0.01).to(bf) if case["bias"] else None
    st["b_up"] = _normal(g, F, std=0.01).to(bf) if case["bias"] else None
    if op == "ffn":
        st["sm_h"] = torch.exp(_normal(g, F, std=0.5)) if case["smooth"] else None
        st["w_down"] = _weights(g, K, F, st["sm_h"])
        st["b_down"] = _normal(g, K, std=0.01).to(bf) if case["bias"] else None
    return st


# ----------------------------------------------------------- plain forms

def _spread(s, n, axis):
    """Each scale for the 128 (the last ones fewer) places that share it."""
    return s.repeat_interleave(BLOCK, axis).narrow(axis, 0, n)


def _blockwise(v):
    """v fp32 [M, K] as the values of its e4m3 codes and their scales, one for a row's
    128 channels: [M, K]."""
    M, K = v.shape
    pad = torch.zeros(M, -K % BLOCK, device=v.device)
    s = torch.cat([v, pad], 1).view(M, -1, BLOCK).abs().amax(2) * torch.tensor(1.0 / LARGEST, dtype=torch.float32)
    i = 1.0 / s
    i = torch.where(torch.isfinite(i), i, torch.zeros_like(i))
    return (v * _spread(i, K, 1)).to(torch.float8_e4m3fn).float() * _spread(s, K, 1)


def _deal(w):
    codes, s = w
    return codes.float() * _spread(_spread(s, codes.shape[0], 0), codes.shape[1], 1)


def _product(v, w, b):
    y = v @ _deal(w).t()
    return y if b is None else y + b.float()


def _gelu(y):
    return 0.5 * y * (1 + torch.tanh(GELU_C * (y + 0.044715 * y * y * y)))


def _smoothed(st):
    v = st["x"].float()
    return v if st["sm"] is None else (v * (1.0 / st["sm"])).to(torch.bfloat16).float()


def _unit(v, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)


def _rows(v, M):
    return v.float().repeat_interleave(M // v.shape[0], 0)


def _plain(st):
    op, bf = st["op"], torch.bfloat16
    if op == "norm_linear":
        M = st["M"]
        h = st["x"].float() + _rows(st["gate"], M) * st["y"].float()
        z = _unit(h, st["norm"]) * (1 + _rows(st["scale"], M)) + _rows(st["shift"], M)
        y = _product(_blockwise(z * (1.0 / st["sm"])), st["w"], st["b"])
        return [h.to(bf), (_gelu(y) if st["epilogue"] == "gelu_tanh" else y).to(bf)]
    v = _blockwise(_smoothed(st))
    if op == "linear":
        y = _product(v, st["w"], st["b"])
        return (_gelu(y) if st["epilogue"] == "gelu_tanh" else y).to(bf)
    gate, up = _product(v, st["w_gate"], st["b_gate"]), _product(v, st["w_up"], st["b_up"])
    h = (gate / (1 + torch.exp(-gate)) if st["act"] == "silu" else _gelu(gate)) * up
    if op == "gated":
        return h.to(bf)
    if st["sm_h"] is not None:
        h = h * (1.0 / st["sm_h"])
    return _product(_blockwise(h), st["w_down"], st["b_down"]).to(bf)


# ------------------------------------------------- the package's operators

def _own(st):
    import bit_diffusion_transformer_svdq_amd as K
    op = st["op"]
    if op == "norm_linear":
        h, (codes, scales) = K.gate_norm_modulate(st["x"], st["y"], gate=st["gate"], norm=st["norm"],
                                                  scale=st["scale"], shift=st["shift"], eps=1e-6,
                                                  quantize="fp8", smooth=st["sm"])
        return [h, K.fp8_gemm(codes, scales, *st["w"], st["b"], epilogue=st["epilogue"])]
    codes, scales = K.quantize_act_fp8(st["x"], st["sm"])
    if op == "linear":
        return K.fp8_gemm(codes, scales, *st["w"], st["b"], epilogue=st["epilogue"])
    if op == "gated":
        return K.fp8_gated_gemm(codes, scales, *st["w_gate"], *st["w_up"], st["b_gate"], st["b_up"],
                                activation=st["act"])
    codes, scales = K.fp8_gated_gemm(codes, scales, *st["w_gate"], *st["w_up"], st["b_gate"], st["b_up"],
                                     activation=st["act"], quantize="fp8", smooth=st["sm_h"])
    return K.fp8_gemm(codes, scales, *st["w_down"], st["b_down"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def _weight_bytes(N, K):
    return N * K + 4 * (-(-N // BLOCK)) * (-(-K // BLOCK))


def work(case):
    op, M = case["op"], case["M"]
    if op == "norm_linear":
        B, C, N = case["B"], case["C"], case["N"]
        return {"bytes": 6 * M * C + 6 * B * C + 4 * C + _weight_bytes(N, C) + 2 * N + 2 * M * N,
                "flops": 2 * M * N * C + 12 * M * C}
    K = case["C"] if op == "ffn" else case["K"]
    read = 2 * M * K + (4 * K if case["smooth"] else 0)
    if op == "linear":
        N = case["N"]
        return {"bytes": read + _weight_bytes(N, K) + (2 * N if case["bias"] else 0) + 2 * M * N,
                "flops": 2 * M * N * K}
    F = case["F"]
    read += 2 * _weight_bytes(F, K) + (4 * F if case["bias"] else 0)
    if op == "gated":
        return {"bytes": read + 2 * M * F, "flops": 4 * M * F * K}
    return {"bytes": read + _weight_bytes(K, F) + (4 * F if case["smooth"] else 0) + (2 * K if case["bias"] else 0)
            + 2 * M * K, "flops": 6 * M * F * K}


# ----------------------------------------------------------------- exact

def _exact_e4m3(t):
    """The nearest e4m3 value of fp32 t (ties to the even one), in 64 bits: 3 bits after
    the leading one, steps of 2^-9 below 2^-6."""
    t = t.double()
    e = torch.frexp(t)[1].double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.round(t / step) * step


def _exact_codes(v):
    """v in 64 bits -> its quantized values: scale and reciprocal are the fp32 numbers
    that the definition names."""
    parts = []
    for block in v.split(BLOCK, dim=1):
        s = block.abs().max(dim=1, keepdim=True).values.float() * (torch.ones(1, device=v.device) / LARGEST)
        inv = torch.reciprocal(s)
        inv[torch.isinf(inv)] = 0
        parts.append(_exact_e4m3(block.float() * inv) * s.double())
    return torch.cat(parts, 1)


def _exact_product(v, w, b):
    codes, s = w
    total = torch.zeros(v.shape[0], codes.shape[0], dtype=torch.float64, device=v.device)
    row = torch.arange(codes.shape[0], device=v.device) // BLOCK
    for k, part in enumerate(v.split(BLOCK, dim=1)):
        c = codes[:, k * BLOCK:(k + 1) * BLOCK].double()
        total += torch.matmul(part, c.T) * s[row, k].double().unsqueeze(0)
    return total if b is None else total + b.double()


def _exact_gelu(y):
    return y / (1 + torch.exp(-2 * GELU_C * (y + 0.044715 * y ** 3)))


def exact(case, seed):
    st = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "norm_linear":
        at = torch.arange(M, device="cuda") // (M // case["B"])
        h = st["x"].double() + st["gate"].double()[at] * st["y"].double()
        d = h - (h.sum(-1, keepdim=True) / h.shape[-1] if case["norm"] == "layer" else 0.0)
        z = d / ((d ** 2).sum(-1, keepdim=True) / h.shape[-1] + 1e-6).sqrt()
        z = z + z * st["scale"].double()[at] + st["shift"].double()[at]
        y = _exact_product(_exact_codes(z / st["sm"].double()), st["w"], st["b"])
        return [h, _exact_gelu(y) if case["epilogue"] == "gelu_tanh" else y]
    v = st["x"].double()
    if st["sm"] is not None:
        v = (st["x"].float() * torch.reciprocal(st["sm"])).bfloat16().double()
    v = _exact_codes(v)
    if op == "linear":
        y = _exact_product(v, st["w"], st["b"])
        return _exact_gelu(y) if case["epilogue"] == "gelu_tanh" else y
    gate, up = _exact_product(v, st["w_gate"], st["b_gate"]), _exact_product(v, st["w_up"], st["b_up"])
    h = up * (gate * torch.sigmoid(gate) if case["act"] == "silu" else _exact_gelu(gate))
    if op == "gated":
        return h
    if st["sm_h"] is not None:
        h = h / st["sm_h"].double()
    return _exact_product(_exact_codes(h), st["w_down"], st["b_down"])
