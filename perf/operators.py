"""Cases of the operators around the ConvRot layer, and their plain forms.

Three operators, as a video DiT block calls them around its linear layers:

- "norm": h = x + residual, RMS norm, ConvRot256 rotation and row-scaled S8 codes held as FP16 (rms_norm_quant);
- "rope": RMS norm of each head of q and k and rotary positions with several axes (qk_norm_rope);
- "gemm": the integer product of two operands of codes, with bias, activation, channel gate and residual in its
  epilogue (gemm_fused).

`own` False computes them in elementary torch operations in 32 bits, `own` True calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 256
EPS = 1e-6
FEW = 64            # most tokens that one-byte weight codes are multiplied with directly

# widths of the DiT whose layers this library runs (hidden, heads x head width, FFN, packed qkv), and its token count
TOKENS, HIDDEN, FFN, QKV, FC1 = 19989, 5376, 14336, 21504, 28672


def padded(K):
    return -(-K // BLOCK) * BLOCK


def listed():
    return [
        # the block's second norm over a whole video: attention output plus residual stream
        {"name": "norm video", "op": "norm", "M": TOKENS, "K": HIDDEN, "dtype": "bf16", "residual": True},
        # one token (an appended one, or a conditioning vector): latency
        {"name": "norm one token", "op": "norm", "M": 1, "K": HIDDEN, "dtype": "fp16", "residual": True},
        # a width that is no multiple of the rotation block, FP32 stream, the first norm (nothing to add)
        {"name": "norm ragged", "op": "norm", "M": 4097, "K": 5000, "dtype": "fp32", "residual": False},
        # q and k of the packed qkv output over a whole video, time x height x width
        {"name": "rope video", "op": "rope", "M": TOKENS, "heads_q": 56, "heads_k": 56, "D": 128, "dtype": "bf16",
         "p0": 16, "p1": 24, "p2": 24, "gh": 36, "gw": 64, "interleaved": False, "norm": True},
        # one token
        {"name": "rope one token", "op": "rope", "M": 1, "heads_q": 56, "heads_k": 56, "D": 128, "dtype": "bf16",
         "p0": 16, "p1": 24, "p2": 24, "gh": 36, "gw": 64, "interleaved": False, "norm": True},
        # an image (height x width) with shared k heads, interleaved pairs, a head partly rotated, no norm
        {"name": "rope image", "op": "rope", "M": 4097, "heads_q": 32, "heads_k": 8, "D": 96, "dtype": "fp16",
         "p0": 20, "p1": 20, "p2": 0, "gh": 64, "gw": 65, "interleaved": True, "norm": False},
        # FFN down, gated and added to the residual stream, a whole video
        {"name": "gemm down video", "op": "gemm", "M": TOKENS, "K": FFN, "N": HIDDEN, "codes": "f16", "out": "bf16",
         "bias": False, "act": "none", "gate": True, "residual": True},
        # FFN up with bias and GELU, part of a video
        {"name": "gemm up", "op": "gemm", "M": 8192, "K": HIDDEN, "N": FC1, "codes": "f16", "out": "bf16",
         "bias": True, "act": "gelu_tanh", "gate": False, "residual": False},
        # ragged rows and columns, FP32 output
        {"name": "gemm ragged", "op": "gemm", "M": 4097, "K": 5000, "N": 21500, "codes": "f16", "out": "fp32",
         "bias": True, "act": "silu", "gate": False, "residual": False},
        # a prompt's text tokens through the output projection
        {"name": "gemm text", "op": "gemm", "M": 256, "K": HIDDEN, "N": HIDDEN, "codes": "f16", "out": "bf16",
         "bias": True, "act": "none", "gate": True, "residual": True},
        # a few tokens, weights resident as the GEMM's FP16 codes
        {"name": "gemm few tokens", "op": "gemm", "M": 16, "K": FFN, "N": HIDDEN, "codes": "f16", "out": "bf16",
         "bias": False, "act": "none", "gate": False, "residual": True},
        # one token, weights resident at one byte per code
        {"name": "gemm one token", "op": "gemm", "M": 1, "K": HIDDEN, "N": QKV, "codes": "s8", "out": "bf16",
         "bias": True, "act": "silu", "gate": False, "residual": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "gemm", "gemm"])
    if op == "norm":
        K = _log(rng, 64, 20480)
        M = min(_log(rng, 1, 20000), TOKENS * HIDDEN // K)
        return {"op": "norm", "M": M, "K": K, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "residual": rng.random() < 0.6}
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128])
        axes = rng.choice([1, 2, 3])
        pairs = D // 2 if rng.random() < 0.7 else D // 4
        cut = sorted(rng.sample(range(1, pairs), axes - 1)) + [pairs]
        parts = [b - a for a, b in zip([0] + cut, cut)] + [0, 0]
        heads_k = _log(rng, 1, 56)
        heads_q = heads_k * rng.choice([1, 1, max(1, 56 // heads_k)])
        return {"op": "rope", "M": _log(rng, 1, 19989), "heads_q": heads_q, "heads_k": heads_k, "D": D,
                "dtype": rng.choice(["bf16", "fp16"]), "p0": parts[0], "p1": parts[1], "p2": parts[2],
                "gh": _log(rng, 1, 90), "gw": _log(rng, 1, 120), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.6}
    few = rng.random() < 0.4
    M = _log(rng, 1, FEW) if few else _log(rng, FEW + 1, 20000)
    K, N = _log(rng, 256, 20480), _log(rng, 256, FC1)
    most = TOKENS * FFN * HIDDEN
    if M * padded(K) * N > most:
        N = max(1, most // (M * padded(K)))
    residual = rng.random() < 0.5
    return {"op": "gemm", "M": M, "K": K, "N": N, "codes": rng.choice(["s8", "f16"]) if few else "f16",
            "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5,
            "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
            "gate": residual and rng.random() < 0.5, "residual": residual}


def _pairs(case):
    return [p for p in (case["p0"], case["p1"], case["p2"]) if p > 0]


def _inv_freq(pairs, theta=10000.0):
    """Radians per unit of position of every rotated pair: each axis spans its own frequencies."""
    return [theta ** (-j / p) for p in pairs for j in range(p)]


def _rotation():
    """The 256-point rotation: the Sylvester matrix, (-1) ** (bits that row and column share), over 16."""
    i = torch.arange(BLOCK)
    shared = ((i[:, None] & i)[:, :, None] >> torch.arange(8) & 1).sum(2)
    return (1.0 - 2.0 * (shared % 2)) / 16.0


def _codes(rows, cols, kind, g):
    """Rows of codes as the quantisers leave them: near normal after the rotation, the largest at 127."""
    q = torch.randn(rows, cols, generator=g, device="cuda").mul_(30.0).round_().clamp_(-127, 127)
    return q.to(torch.int8 if kind == "s8" else torch.float16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def rand(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        M, K, dt = case["M"], case["K"], DTYPES[case["dtype"]]
        x = rand(M, K)
        x[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device=dev)] *= 20.0     # outlier channels
        s["x"] = x.to(dt)
        s["residual"] = rand(M, K, dtype=dt, std=2.0) if case["residual"] else None
        s["h"] = torch.empty(M, K, dtype=dt, device=dev) if case["residual"] else None
        s["weight"] = 1.0 + 0.1 * rand(K)
        s["rot"] = _rotation().to(device=dev, dtype=torch.float32)
        s["codes"] = torch.empty(M, padded(K), dtype=torch.float16, device=dev)
        s["scale"] = torch.empty(M, dtype=torch.float32, device=dev)
    elif case["op"] == "rope":
        M, D, Hq, Hk, dt = case["M"], case["D"], case["heads_q"], case["heads_k"], DTYPES[case["dtype"]]
        qkv = rand(M, (Hq + 2 * Hk) * D, dtype=dt)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        s["q_out"] = torch.empty(M, Hq, D, dtype=dt, device=dev)
        s["k_out"] = torch.empty(M, Hk, D, dtype=dt, device=dev)
        pairs = _pairs(case)
        first = torch.randint(0, 512, (1,), generator=g, device=dev)
        i = torch.arange(M, device=dev)
        gh, gw = case["gh"], case["gw"]
        where = {1: [i], 2: [i // gw, i % gw], 3: [i // (gh * gw), i // gw % gh, i % gw]}[len(pairs)]
        pos = torch.stack(where, 1)
        pos[:, 0] += first
        s["pos"] = pos.to(torch.int32)
        s["inv_freq"] = torch.tensor(_inv_freq(pairs), dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor([a for a, p in enumerate(pairs) for _ in range(p)], device=dev)
        s["pairs"] = pairs
        s["q_weight"] = 1.0 + 0.1 * rand(D) if case["norm"] else None
        s["k_weight"] = 1.0 + 0.1 * rand(D) if case["norm"] else None
    else:
        M, N, Kp, dt = case["M"], case["N"], padded(case["K"]), DTYPES[case["out"]]
        s["a"], s["w"] = _codes(M, Kp, case["codes"], g), _codes(N, Kp, case["codes"], g)
        s["sa"] = 0.03 * (1.0 + 0.2 * torch.rand(M, generator=g, device=dev))
        s["sw"] = 0.03 / math.sqrt(Kp) * (1.0 + 0.2 * torch.rand(N, generator=g, device=dev))
        s["bias"] = rand(N, std=0.5) if case["bias"] else None
        s["gate"] = rand(N) if case["gate"] else None
        s["residual"] = rand(M, N, dtype=dt, std=2.0) if case["residual"] else None
        s["out"] = torch.empty(M, N, dtype=dt, device=dev)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "rope": _own_rope, "gemm": _own_gemm}[op](s)
    return {"norm": _plain_norm, "rope": _plain_rope, "gemm": _plain_gemm}[op](s)


# ---------------------------------------------------------------- the library's calls
def _own_norm(s):
    import rotated_w4a8_int8_gb300 as cr
    cr.rms_norm_quant(s["x"], s["case"]["K"], s["codes"], s["scale"], residual=s["residual"], h=s["h"],
                      weight=s["weight"], eps=EPS)
    return {"codes": s["codes"], "scale": s["scale"], **({"h": s["h"]} if s["h"] is not None else {})}


def _own_rope(s):
    import rotated_w4a8_int8_gb300 as cr
    cr.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["pairs"], s["q_out"], s["k_out"],
                    q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["case"]["interleaved"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_gemm(s):
    import rotated_w4a8_int8_gb300 as cr
    act = {"none": cr.ACT_NONE, "relu": cr.ACT_RELU, "silu": cr.ACT_SILU, "gelu": cr.ACT_GELU,
           "gelu_tanh": cr.ACT_GELU_TANH}[s["case"]["act"]]
    cr.gemm_fused(s["a"], s["sa"], s["w"], s["sw"], s["out"], bias=s["bias"], act=act, gate=s["gate"],
                  residual=s["residual"])
    return s["out"]


# ---------------------------------------------------------------- plain forms
def _plain_norm(s):
    x, M, K = s["x"], s["case"]["M"], s["case"]["K"]
    out = {}
    if s["residual"] is not None:
        out["h"] = x = (x.float() + s["residual"].float()).to(x.dtype)
    h = x.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
    Kp = padded(K)
    v = torch.zeros(M, Kp, device=y.device)
    v[:, :K] = y
    v = (v.view(M, Kp // BLOCK, BLOCK) @ s["rot"]).view(M, Kp)
    scale = v.abs().amax(1) / 127.0
    r = 1.0 / scale
    dead = (scale == 0) | torch.isinf(r)
    scale, r = torch.where(dead, 0.0, scale), torch.where(dead, 0.0, r)
    out["codes"] = (v * r[:, None]).round().clamp(-127, 127).to(torch.float16)
    out["scale"] = scale
    return out


def _plain_heads(x, weight, cos, sin, interleaved):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(2, keepdim=True) + EPS) * weight
    P = cos.shape[2]
    if interleaved:
        a, b = y[:, :, 0:2 * P:2], y[:, :, 1:2 * P:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = y[:, :, :P], y[:, :, P:2 * P]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([turned, y[:, :, 2 * P:]], 2).to(x.dtype)


def _plain_rope(s):
    angle = (s["pos"].float()[:, s["axis"]] * s["inv_freq"].float())[:, None, :]
    cos, sin, il = torch.cos(angle), torch.sin(angle), s["case"]["interleaved"]
    return {"q": _plain_heads(s["q"], s["q_weight"], cos, sin, il), "k": _plain_heads(s["k"], s["k_weight"], cos, sin, il)}


def _plain_gemm(s):
    y = (s["a"].float() @ s["w"].float().T) * s["sa"][:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"]
    act = s["case"]["act"]
    if act == "relu":
        y = torch.where(y < 0, 0.0, y)
    elif act == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["gate"] is not None:
        y = y * s["gate"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["out"].dtype)


# ---------------------------------------------------------------- work and definition
def work(case):
    M = case["M"]
    if case["op"] == "norm":
        K, e = case["K"], BYTES[case["dtype"]]
        # x (and the residual in, the sum out), the weight, the FP16 codes with their padding, the scales
        return {"bytes": M * K * e * (3 if case["residual"] else 1) + 4 * K + M * padded(K) * 2 + 4 * M,
                "flops": 14 * M * padded(K)}
    if case["op"] == "rope":
        n = M * (case["heads_q"] + case["heads_k"]) * case["D"]
        return {"bytes": 2 * n * BYTES[case["dtype"]] + 4 * M * len(_pairs(case)), "flops": (7 if case["norm"] else 3) * n}
    N, Kp = case["N"], padded(case["K"])
    e = BYTES[case["out"]]
    return {"bytes": (M + N) * Kp * (1 if case["codes"] == "s8" else 2) + M * N * e * (2 if case["residual"] else 1)
            + 4 * M + 4 * N * (1 + case["bias"] + case["gate"]), "flops": 2 * M * N * Kp}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        M, K, Kp = case["M"], case["K"], padded(case["K"])
        x = s["x"].to(f64)
        res = {}
        if s["residual"] is not None:
            x = (x + s["residual"].to(f64)).to(s["x"].dtype).to(f64)
            res["h"] = x
        y = torch.zeros(M, Kp, dtype=f64, device=x.device)
        y[:, :K] = x / (x.square().sum(1, keepdim=True) / K + EPS).sqrt() * s["weight"].to(f64)
        y = y.view(-1, BLOCK)
        step = 1
        while step < BLOCK:                       # the transform's butterflies, stage by stage
            y = y.view(-1, BLOCK // (2 * step), 2, step)
            y = torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2)
            step *= 2
        y = y.reshape(M, Kp) / 16.0
        scale = y.abs().amax(1) / 127.0
        res["codes"] = torch.where(scale[:, None] > 0, (y / scale[:, None]).round(), 0.0)
        res["scale"] = scale
        return res
    if case["op"] == "rope":
        phi = torch.empty(case["M"], 0, dtype=f64, device="cuda")
        at = 0
        for a, p in enumerate(s["pairs"]):
            phi = torch.cat([phi, s["pos"][:, a:a + 1].to(f64) * s["inv_freq"][at:at + p]], 1)
            at += p
        turn = torch.polar(torch.ones_like(phi), phi)[:, None, :]

        def one(x, w):
            x = x.to(f64)
            if w is not None:
                x = x / (x.square().sum(2, keepdim=True) / x.shape[2] + EPS).sqrt() * w.to(f64)
            x = x.clone()
            ev, od = (slice(0, 2 * at, 2), slice(1, 2 * at, 2)) if case["interleaved"] else (slice(0, at), slice(at, 2 * at))
            z = torch.complex(x[:, :, ev], x[:, :, od]) * turn
            x[:, :, ev], x[:, :, od] = z.real, z.imag
            return x
        return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}
    if 2.0 * case["M"] * case["N"] * padded(case["K"]) > 8e12:
        return None
    v = torch.matmul(s["a"].to(f64), s["w"].to(f64).t())
    v *= s["sa"].to(f64).unsqueeze(1)
    v *= s["sw"].to(f64)
    if s["bias"] is not None:
        v += s["bias"].to(f64)
    c = math.sqrt(2.0 / math.pi)
    f = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "silu": lambda t: t * torch.sigmoid(t),
         "gelu": lambda t: t * torch.special.ndtr(t),
         "gelu_tanh": lambda t: t * torch.sigmoid(2.0 * c * (t + 0.044715 * t ** 3))}[case["act"]]
    v = f(v)
    if s["gate"] is not None:
        v *= s["gate"].to(f64)
    if s["residual"] is not None:
        v += s["residual"].to(f64)
    return v
