"""What is measured of the diffusion-transformer block operators: the 8-bit linear
(per-token, per-channel scales), the gated residual norms and the rotary
positions with several axes.

``run`` computes a case in its plain form (elementary torch operations in
32 bits, 64 where 32 lose what matters) or, where ``own`` is true, with the
package's operators.  Sizes follow a 12B-class diffusion transformer at 1024²
(hidden 3072, 4096 image and 512 text tokens, heads of 128, rotary axes
16 + 56 + 56) and generic smaller and odd ones.
"""
from __future__ import annotations

import math

import torch

own = False

GELU_C = math.sqrt(2.0 / math.pi)


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one conditioning vector through an embedder's second linear: latency
        dict(name="linear 1 token", op="linear", M=1, K=3072, N=3072, smooth=False, bias=True, epilogue="none"),
        # a patch sequence of an odd picture through a mid-size up-projection
        dict(name="linear 1333 tokens", op="linear", M=1333, K=1920, N=7744, smooth=True, bias=True,
             epilogue="gelu_tanh"),
        # the MLP up-projection of all 4608 tokens of a 1024² image
        dict(name="linear 4608 tokens", op="linear", M=4608, K=3072, N=12288, smooth=True, bias=True,
             epilogue="gelu_tanh"),
        # the final norm of a few pooled rows: latency
        dict(name="norm 3 rows", op="norm", M=3, B=3, C=1536, stream="bf16", block=False, post="none",
             norm="layer", weight=False),
        # after attention: gated residual, norm and modulation before the MLP, one image
        dict(name="norm 4608 rows", op="norm", M=4608, B=1, C=3072, stream="bf16", block=True, post="none",
             norm="layer", weight=False),
        # norms on both sides of the block, residual stream in fp32, two pictures of an odd size
        dict(name="sandwich 2 x 4173 rows", op="norm", M=8346, B=2, C=2304, stream="fp32", block=True, post="rms",
             norm="rms", weight=True),
        # norm into 8 bits and the up-projection of 64 tokens
        dict(name="norm + linear 64", op="norm_linear", M=64, B=1, C=3072, N=12288, epilogue="gelu_tanh"),
        # norm into 8 bits and the QKV projection of the text stream
        dict(name="norm + linear 512", op="norm_linear", M=512, B=1, C=3072, N=9216, epilogue="none"),
        # the tables of a step's 4608 positions (read by the fused QKV epilogue)
        dict(name="tables 4608", op="tables", M=4608, axes="16,56,56", spectrum="axis", far=False),
        # a handful of new tokens, grouped heads: latency
        dict(name="rope 7 tokens", op="rope", M=7, P=7, Hq=16, Hk=2, D=128, axes="64,64", spectrum="axis",
             layout="pairs", norm=False, fused=False, far=True),
        # Q and K of the fused QKV output of a 1024² image, head norm first
        dict(name="rope 4608 tokens", op="rope", M=4608, P=4608, Hq=24, Hk=24, D=128, axes="16,56,56",
             spectrum="axis", layout="pairs", norm=True, fused=True, far=False),
        # two clips that share their (time, height, width) positions
        dict(name="rope 2 x 16380 tokens", op="rope", M=32760, P=16380, Hq=12, Hk=12, D=128, axes="44,42,42",
             spectrum="axis", layout="halves", norm=False, fused=False, far=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "norm", "norm_linear", "rope", "rope", "tables"])
    if op == "linear":
        K, N, M = 64 * _log(rng, 4, 192), 64 * _log(rng, 2, 192), _log(rng, 1, 4608)
        M = max(1, min(M, 4608 * 3072 * 12288 // (K * N)))
        return dict(op=op, M=M, K=K, N=N, smooth=rng.random() < 0.5, bias=rng.random() < 0.7,
                    epilogue=rng.choice(["none", "gelu_tanh"]))
    if op == "norm":
        B = rng.choice([1, 1, 2, 3])
        C = 8 * _log(rng, 16, 640)
        S = max(1, _log(rng, 1, 24_000_000 // (C * B)))
        block = rng.random() < 0.7
        return dict(op=op, M=B * S, B=B, C=C, stream=rng.choice(["bf16", "fp32"]), block=block,
                    post=rng.choice(["none", "rms", "layer"]) if block else "none",
                    norm=rng.choice(["layer", "rms"]), weight=rng.random() < 0.5)
    if op == "norm_linear":
        C, N, M = 64 * _log(rng, 4, 64), 64 * _log(rng, 2, 192), _log(rng, 1, 4096)
        M = min(M, 4608 * 3072 * 12288 // (C * N))
        return dict(op=op, M=M, B=1, C=C, N=N, epilogue=rng.choice(["none", "gelu_tanh"]))
    D = rng.choice([64, 80, 96, 128])
    half = D // 2
    parts = sorted(rng.sample(range(4, half - 3, 4), rng.choice([1, 2])))
    cuts = [0] + parts + [half]
    axes = ",".join(str(2 * (b - a)) for a, b in zip(cuts, cuts[1:]))
    if op == "tables":
        return dict(op=op, M=_log(rng, 1, 60000), axes=axes, spectrum=rng.choice(["axis", "shared"]),
                    far=rng.random() < 0.3)
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4])
    B = rng.choice([1, 1, 2])
    P = max(1, _log(rng, 1, 50_000_000 // (B * (Hq + Hk) * D)))
    fused = rng.random() < 0.5
    return dict(op=op, M=B * P, P=P, Hq=Hq, Hk=Hk, D=D, axes=axes, spectrum=rng.choice(["axis", "shared"]),
                layout=rng.choice(["pairs", "halves"]), norm=rng.random() < 0.5, fused=fused,
                far=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activations(g, M, C):
    """Unit normal rows with 1 % of the channels 30 times as large."""
    x = _normal(g, M, C)
    loud = torch.randperm(C, generator=g, device="cuda")[:max(1, C // 100)]
    x[:, loud] *= 30.0
    return x


def _linear_weights(g, N, K, smooth):
    """8-bit codes and channel scales of N(0, 0.02) weights, smoothing moved into them."""
    w = _normal(g, N, K, std=0.02)
    if smooth is not None:
        w = w * smooth
    s = w.abs().amax(1) / 127.0
    return torch.round(w / s[:, None]).to(torch.int8), s


def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _positions(g, case, rows):
    """Grid positions (time, height, width ...) of a picture or clip; whole
    numbers or, for the far ones, a long way from the origin."""
    n = len(_axes(case))
    side = max(1, int(round(rows ** (1.0 / max(1, n - 1)))))
    i = torch.arange(rows, device="cuda")
    cols = [(i // side ** (n - 1 - a)) % max(side, 1) if a else i // side ** (n - 1) for a in range(n)]
    pos = torch.stack(cols, 1).to(torch.float32)
    shift = torch.randint(0, 16, (1, n), generator=g, device="cuda").float()
    if case["far"]:
        shift = shift + torch.randint(100_000, 1_000_000, (1, n), generator=g, device="cuda").float()
    return (pos + shift).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, st = case["op"], dict(case)
    bf = torch.bfloat16
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        x = _activations(g, M, K).to(bf)
        st["x"] = x
        # the smoothing vector of the layer: larger where activations are
        sm = (x.float().abs().amax(0).clamp(min=1e-2) / 0.08).sqrt() if case["smooth"] else None
        st["smooth_v"] = sm
        st["w_codes"], st["w_scales"] = _linear_weights(g, N, K, sm)
        st["b"] = _normal(g, N, std=0.01).to(bf) if case["bias"] else None
    elif op in ("norm", "norm_linear"):
        M, B, C = case["M"], case["B"], case["C"]
        x = _activations(g, M, C)
        st["x"] = x if case.get("stream") == "fp32" else x.to(bf)
        blk = case.get("block", True)
        st["y"] = _normal(g, M, C, std=0.7).to(bf) if blk else None
        # one projection gives every vector of the block: strided chunks of it
        mod = _normal(g, B, 3 * C, std=0.3).to(bf)
        st["gate"], st["scale"], st["shift"] = mod[:, :C], mod[:, C:2 * C], mod[:, 2 * C:]
        if not blk:
            st["gate"] = None
        st["w_norm"] = (1 + _normal(g, C, std=0.1)).to(bf) if case.get("weight") else None
        st["w_post"] = (1 + _normal(g, C, std=0.1)).to(bf) if case.get("post", "none") != "none" else None
        if op == "norm_linear":
            sm = torch.exp(_normal(g, C, std=0.3))
            st["smooth_v"] = sm
            st["w_codes"], st["w_scales"] = _linear_weights(g, case["N"], C, sm)
            st["b"] = _normal(g, case["N"], std=0.01).to(bf)
    elif op == "tables":
        st["pos"] = _positions(g, case, case["M"])
    else:
        M, Hq, Hk, D = case["M"], case["Hq"], case["Hk"], case["D"]
        if case["fused"]:  # thirds of the projection's output, as it leaves the linear
            qkv = _normal(g, M, (Hq + 2 * Hk) * D, std=1.5).to(bf)
            st["q"] = qkv[:, :Hq * D].view(M, Hq, D)
            st["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D)
        else:
            st["q"] = _normal(g, M, Hq, D, std=1.5).to(bf)
            st["k"] = _normal(g, M, Hk, D, std=1.5).to(bf)
        st["pos"] = _positions(g, case, case["P"])
        st["qn"] = (1 + _normal(g, D, std=0.1)).to(bf) if case["norm"] else None
        st["kn"] = (1 + _normal(g, D, std=0.1)).to(bf) if case["norm"] else None
    return st


# ----------------------------------------------------------- plain forms

def _quantize(v):
    """Per-token 8-bit codes (as fp32) and scales of v fp32 [M, K]."""
    s = v.abs().amax(1) / 127.0
    i = 1.0 / s
    # the product is exact in 64 bits: a value next to a border keeps its side
    q = torch.round(v.double() * i.double()[:, None]).clamp(-127, 127).float()
    return torch.where(torch.isfinite(i)[:, None], q, torch.zeros_like(q)), s


def _product(q, s, st):
    acc = q @ st["w_codes"].float().t()
    y = acc * (s[:, None] * st["w_scales"])
    if st["b"] is not None:
        y = y + st["b"].float()
    if st["epilogue"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(GELU_C * (y + 0.044715 * y * y * y)))
    return y.to(torch.bfloat16)


def _norm(v, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)


def _rows(v, M):
    return v.float().repeat_interleave(M // v.shape[0], 0)


def _norm_rows(st):
    """(h in fp32, z in fp32) of the gated residual and the modulated norm."""
    M, h = st["M"], st["x"].float()
    if st["y"] is not None:
        u = st["y"].float()
        if st.get("post", "none") != "none":
            u = _norm(u, st["post"]) * st["w_post"].float()
        h = h + _rows(st["gate"], M) * u
    n = _norm(h, st.get("norm", "layer"))
    if st["w_norm"] is not None:
        n = n * st["w_norm"].float()
    return h, n * (1 + _rows(st["scale"], M)) + _rows(st["shift"], M)


def _angles(st, rows):
    """cos and sin, fp32 [rows, R/2]; the angles of far positions need 64 bits."""
    axes = _axes(st)
    R, pos = sum(axes), st["pos"].double()
    parts, first = [], 0
    for a, d in enumerate(axes):
        j = torch.arange(d // 2, device="cuda", dtype=torch.float64)
        e = 2 * j / d if st["spectrum"] == "axis" else 2 * (first + j) / R
        parts.append(pos[:, a:a + 1] * (10000.0 ** -e))
        first += d // 2
    t = torch.cat(parts, 1).repeat(rows // pos.shape[0], 1)
    return t.cos().float(), t.sin().float()


def _turn(v, w, c, s, st):
    v = v.float()
    if w is not None:
        v = v * torch.rsqrt((v * v).mean(2, keepdim=True) + 1e-6) * w.float()
    R = 2 * c.shape[1]
    c, s, t = c[:, None], s[:, None], v[..., :R]
    if st["layout"] == "pairs":
        a, b = t[..., 0::2], t[..., 1::2]
        out = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(2)
    else:
        a, b = t[..., :R // 2], t[..., R // 2:]
        out = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([out, v[..., R:]], -1).to(torch.bfloat16)


def _plain(st):
    op, bf = st["op"], torch.bfloat16
    if op == "linear":
        v = st["x"].float()
        if st["smooth_v"] is not None:
            v = (v * (1.0 / st["smooth_v"])).to(bf).float()
        return _product(*_quantize(v), st)
    if op == "norm":
        h, z = _norm_rows(st)
        return ([h.to(st["x"].dtype)] if st["y"] is not None else []) + [z.to(bf)]
    if op == "norm_linear":
        h, z = _norm_rows(st)
        return [h.to(bf), _product(*_quantize(z * (1.0 / st["smooth_v"])), st)]
    if op == "tables":
        return list(_angles(st, st["M"]))
    c, s = _angles(st, st["M"])
    return [_turn(st["q"], st["qn"], c, s, st), _turn(st["k"], st["kn"], c, s, st)]


# ------------------------------------------------- the package's operators

def _own(st):
    import bit_diffusion_transformer_svdq_amd as K
    op = st["op"]
    if op == "linear":
        codes, scales = K.quantize_act_int8(st["x"], st["smooth_v"])
        return K.w8a8_gemm(codes, scales, st["w_codes"], st["w_scales"], st["b"], epilogue=st["epilogue"])
    if op == "norm":
        h, z = K.gate_norm_modulate(st["x"], st["y"], post_norm=st["post"], post_weight=st["w_post"],
                                    gate=st["gate"], norm=st["norm"], weight=st["w_norm"], scale=st["scale"],
                                    shift=st["shift"], eps=1e-6)
        return [z] if h is None else [h, z]
    if op == "norm_linear":
        h, (codes, scales) = K.gate_norm_modulate(st["x"], st["y"], gate=st["gate"], norm="layer",
                                                  scale=st["scale"], shift=st["shift"], eps=1e-6,
                                                  quantize="int8", smooth=st["smooth_v"])
        return [h, K.w8a8_gemm(codes, scales, st["w_codes"], st["w_scales"], st["b"], epilogue=st["epilogue"])]
    if op == "tables":
        return list(K.rope_axes_tables(st["pos"], _axes(st), theta=10000.0, spectrum=st["spectrum"]))
    return list(K.rope_axes(st["q"], st["k"], st["pos"], _axes(st), theta=10000.0, spectrum=st["spectrum"],
                            layout=st["layout"], q_norm=st["qn"], k_norm=st["kn"], eps=1e-6))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def work(case):
    op, M = case["op"], case["M"]
    if op == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * M * K + (4 * K if case["smooth"] else 0) + N * K + 4 * N + (2 * N if case["bias"] else 0)
                + 2 * M * N, "flops": 2 * M * N * K}
    if op == "norm":
        C, e = case["C"], 4 if case["stream"] == "fp32" else 2
        rows = e * C + (2 * C + e * C if case["block"] else 0) + 2 * C
        vecs = 2 * C * ((3 if case["block"] else 2) * case["B"] + bool(case["weight"]) + (case["post"] != "none"))
        return {"bytes": M * rows + vecs, "flops": 12 * M * C}
    if op == "norm_linear":
        C, N = case["C"], case["N"]
        return {"bytes": 6 * M * C + 6 * C + 4 * C + N * C + 6 * N + 2 * M * N, "flops": 2 * M * N * C + 12 * M * C}
    axes = [int(a) for a in case["axes"].split(",")]
    if op == "tables":
        return {"bytes": 4 * M * (len(axes) + sum(axes)), "flops": 20 * M * sum(axes)}
    n = M * (case["Hq"] + case["Hk"]) * case["D"]
    return {"bytes": 4 * n + 4 * case["P"] * len(axes) + (4 * case["D"] if case["norm"] else 0),
            "flops": (8 if case["norm"] else 4) * n}


# ----------------------------------------------------------------- exact

def _exact_linear(v, case, st):
    """y in fp64 from v (fp64 [M, K]): the token scale is the fp32 quotient the
    definition names, the code the nearest whole number."""
    s = (v.abs().max(dim=1).values.float() / 127).double()
    inv = (1 / s.float()).double()
    q = torch.clamp((v * inv.unsqueeze(1)).round(), min=-127, max=127)
    y = torch.matmul(q, st["w_codes"].double().T) * s.unsqueeze(1) * st["w_scales"].double().unsqueeze(0)
    if st["b"] is not None:
        y += st["b"].double()
    if case["epilogue"] == "gelu_tanh":
        y = y / (1 + torch.exp(-2 * GELU_C * (y + 0.044715 * y ** 3)))
    return y


def _exact_unit(v, kind):
    mean = v.sum(-1, keepdim=True) / v.shape[-1] if kind == "layer" else 0.0
    d = v - mean
    return d / ((d ** 2).sum(-1, keepdim=True) / v.shape[-1] + 1e-6).sqrt()


def exact(case, seed):
    st = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "linear":
        v = st["x"].double()
        if st["smooth_v"] is not None:
            mu = torch.reciprocal(st["smooth_v"])
            v = (st["x"].float() * mu).bfloat16().double()
        return _exact_linear(v, case, st)
    if op in ("norm", "norm_linear"):
        def per_row(t):
            return t.double()[torch.arange(M, device="cuda") // (M // case["B"])]
        h = st["x"].double()
        if st["y"] is not None:
            u = st["y"].double()
            if case.get("post", "none") != "none":
                u = _exact_unit(u, case["post"]) * st["w_post"].double()
            h = h + per_row(st["gate"]) * u
        z = _exact_unit(h, case.get("norm", "layer"))
        if st["w_norm"] is not None:
            z = z * st["w_norm"].double()
        z = z + z * per_row(st["scale"]) + per_row(st["shift"])
        if op == "norm_linear":
            return [h, _exact_linear(z / st["smooth_v"].double(), case, st)]
        return ([h] if st["y"] is not None else []) + [z]
    # the turn as a product of complex numbers
    axes = _axes(case)
    owner = torch.tensor([a for a, d in enumerate(axes) for _ in range(d // 2)], device="cuda")
    if case["spectrum"] == "axis":
        rate = [math.exp(-2.0 * j / d * math.log(10000.0)) for d in axes for j in range(d // 2)]
    else:
        rate = [math.exp(-2.0 * i / sum(axes) * math.log(10000.0)) for i in range(sum(axes) // 2)]
    angle = st["pos"].double()[:, owner] * torch.tensor(rate, dtype=torch.float64, device="cuda")
    unit = torch.polar(torch.ones_like(angle), angle)
    if op == "tables":
        return [unit.real.clone(), unit.imag.clone()]
    unit = unit[torch.arange(M, device="cuda") % case["P"]].unsqueeze(1)
    R, out = sum(axes), []
    for v, w in ((st["q"], st["qn"]), (st["k"], st["kn"])):
        v = v.double()
        if w is not None:
            v = v / (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + 1e-6).sqrt() * w.double()
        t = v[..., :R].clone()
        if case["layout"] == "pairs":
            z = torch.view_as_complex(t.reshape(M, -1, R // 2, 2)) * unit
            t = torch.view_as_real(z).reshape(M, -1, R)
        else:
            z = torch.complex(t[..., :R // 2].contiguous(), t[..., R // 2:].contiguous()) * unit
            t = torch.cat((z.real, z.imag), dim=-1)
        out.append(torch.cat((t, v[..., R:]), dim=-1))
    return out
