"""Workloads of the 8-bit serving operators: row quantisation (with or without
a residual addition and RMS norm), the 8-bit linear product and the
mixture-of-experts layer for a few tokens.

``run`` computes each in plain 32-bit torch operations, or, where ``own`` is
true, through the package's entry points.  ``exact`` restates the definitions
in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token's row: the launch is all there is
        {"name": "norm_token", "op": "rows", "M": 1, "K": 4096, "dtype": "bf16", "norm": True,
         "residual": True, "y": False},
        # a prompt's tokens in front of a product; y feeds a router as well
        {"name": "norm_prompt", "op": "rows", "M": 8192, "K": 4096, "dtype": "bf16", "norm": True,
         "residual": True, "y": True},
        # FP32 tokens with rows that are not a multiple of 16
        {"name": "norm_odd_fp32", "op": "rows", "M": 1001, "K": 4092, "dtype": "fp32", "norm": True,
         "residual": False, "y": False},
        # the hidden rows in front of a down product
        {"name": "quantize_hidden", "op": "rows", "M": 2048, "K": 14336, "dtype": "bf16",
         "norm": False, "residual": False, "y": False},
        # one decoded token through an up product
        {"name": "linear_token", "op": "linear", "M": 1, "N": 14336, "K": 4096, "dtype": "bf16",
         "bias": False, "act": "none"},
        # sixteen decoded sequences through a down product
        {"name": "linear_decode_16", "op": "linear", "M": 16, "N": 4096, "K": 14336,
         "dtype": "bf16", "bias": False, "act": "none"},
        # a short prompt or a wide decode batch
        {"name": "linear_skinny_128", "op": "linear", "M": 128, "N": 14336, "K": 4096,
         "dtype": "bf16", "bias": False, "act": "silu"},
        # ragged in every direction, FP32 result, bias and activation
        {"name": "linear_odd_fp32", "op": "linear", "M": 1001, "N": 4092, "K": 4091,
         "dtype": "fp32", "bias": True, "act": "gelu"},
        # a long prompt through an up product
        {"name": "linear_prompt", "op": "linear", "M": 8192, "N": 14336, "K": 4096,
         "dtype": "bf16", "bias": False, "act": "none"},
        # one decoded token, few large experts
        {"name": "moe_token", "op": "moe", "T": 1, "E": 8, "k": 2, "H": 4096, "I": 14336,
         "dtype": "bf16", "renorm": True},
        # sixteen sequences over many small experts: most experts have some token
        {"name": "moe_16_small", "op": "moe", "T": 16, "E": 64, "k": 6, "H": 2048, "I": 1408,
         "dtype": "bf16", "renorm": False},
        # FP32 tokens, odd count of them
        {"name": "moe_fp32", "op": "moe", "T": 5, "E": 16, "k": 4, "H": 1024, "I": 1000,
         "dtype": "fp32", "renorm": True},
    ]


def _size(rng, lo, hi, step):
    """A size spread over the logarithm of [lo, hi]: a multiple of `step`, or
    any whole number one time in four."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.75:
        n = max(step, n // step * step)
    n = min(hi, max(lo, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(("rows", "linear", "linear", "moe"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "rows":
        norm = rng.random() < 0.7
        K = _size(rng, 256, 16384, 64)
        M = min(_size(rng, 1, 8192, 1), (8192 * 14336) // K)
        return {"op": op, "M": M, "K": K, "dtype": dtype, "norm": norm,
                "residual": norm and rng.random() < 0.7, "y": norm and rng.random() < 0.3}
    if op == "linear":
        N, K = _size(rng, 256, 16384, 64), _size(rng, 256, 16384, 64)
        M = min(_size(rng, 1, 8192, 1), (8192 * 14336 * 4096) // (N * K))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "bias": rng.random() < 0.3,
                "act": rng.choice(("none", "none", "relu", "gelu", "silu"))}
    E = rng.choice((4, 8, 16, 32, 60, 64, 128))
    H = _size(rng, 512, 4096, 64)
    most = min(14336, int(1.4e9 / (3 * E * H)))
    inner = _size(rng, 256, max(512, most), 64)
    return {"op": op, "T": _size(rng, 1, 32, 1), "E": E, "k": rng.choice((1, 2, 4)), "H": H,
            "I": inner, "dtype": dtype, "renorm": rng.random() < 0.5}


def _int8(gen, *shape):
    """8-bit values as a row of normal numbers gives them: a deviation of about 32."""
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return v.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(gen, base, *shape):
    return base * (0.5 + torch.rand(shape, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": case}
    if op == "rows":
        M, K = case["M"], case["K"]
        x = normal(M, K)
        # a few channels carry much larger values, as hidden states do
        x[:, :: max(1, K // 7)] *= 8.0
        s["x"] = x.to(dt)
        s["residual"] = (2.0 * normal(M, K)).to(dt) if case["residual"] else None
        s["weight"] = 1.0 + 0.2 * normal(K) if case["norm"] else None
        s["q"] = torch.empty((M, K), device="cuda", dtype=torch.int8)
        s["scale"] = torch.empty(M, device="cuda")
        s["h"] = torch.empty((M, K), device="cuda", dtype=dt) if case["residual"] else None
        s["y"] = torch.empty((M, K), device="cuda", dtype=dt) if case["y"] else None
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"], s["xs"] = _int8(gen, M, K), _scales(gen, 1.0 / 32, M)
        s["wq"], s["ws"] = _int8(gen, N, K), _scales(gen, 1.0 / (32 * math.sqrt(K)), N)
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        s["out"] = torch.empty((M, N), device="cuda", dtype=dt)
    else:
        T, E, H, inner = case["T"], case["E"], case["H"], case["I"]
        s["x"] = normal(T, H).to(dt)
        s["router"] = normal(E, H) / math.sqrt(H)
        s["w_up"], s["s_up"] = _int8(gen, E, 2 * inner, H), _scales(gen, 1.0 / (32 * math.sqrt(H)), E, 2 * inner)
        s["w_down"], s["s_down"] = _int8(gen, E, H, inner), _scales(gen, 1.0 / (32 * math.sqrt(inner)), E, H)
        s["out"] = torch.empty((T, H), device="cuda", dtype=dt)
        s["ids"] = torch.empty((T, case["k"]), device="cuda", dtype=torch.int32)
        s["gates"] = torch.empty((T, case["k"]), device="cuda")
    return s


def _quantize(p):
    """Whole numbers rint(p * 127/max|p|) of each row, and the row's max|p| / 127."""
    m = p.abs().amax(-1, keepdim=True)
    top = torch.full_like(m, 127.0)      # a tensor: dividing by or into a number multiplies by a reciprocal
    q = torch.where(m > 0, torch.round(p * (top / m)), torch.zeros_like(p))
    return q, m / top


def _plain_rows(s):
    case = s["case"]
    x = s["x"].float()
    out = {}
    if case["residual"]:
        x = x + s["residual"].float()
        out["h"] = x.to(s["x"].dtype)
    p = x * s["weight"] if case["norm"] else x
    q, scale = _quantize(p)
    if case["norm"]:
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        scale = scale * r
        if case["y"]:
            out["y"] = (p * r).to(s["x"].dtype)
    out["q"] = q.to(torch.int8)
    out["scale"] = scale[:, 0]
    return out


def _act(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _plain_linear(s):
    v = (s["xq"].float() @ s["wq"].float().T) * s["xs"][:, None] * s["ws"][None, :]
    if s["bias"] is not None:
        v = v + s["bias"]
    return _act(v, s["case"]["act"]).to(s["out"].dtype)


def _plain_moe(s):
    case = s["case"]
    T, E, k, inner = case["T"], case["E"], case["k"], case["I"]
    x = s["x"].float()
    logits = x @ s["router"].T
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    # a stable sort keeps equal gates in index order: ties go to the lowest
    gates, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    gates, ids = gates[:, :k], ids[:, :k]
    if case["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    xq, xs = _quantize(x)
    if T * k < E:      # the picked experts' weights, once for each token
        w_up, s_up = s["w_up"][ids].float(), s["s_up"][ids]                    # (T, k, 2I, H), (T, k, 2I)
        w_down, s_down = s["w_down"][ids].float(), s["s_down"][ids]
        up = torch.matmul(w_up, xq[:, None, :, None])[..., 0] * xs[:, None, :] * s_up
    else:              # every expert on every token
        up = torch.matmul(xq, s["w_up"].float().transpose(1, 2)) * xs * s["s_up"][:, None, :]
    g, u = up[..., :inner], up[..., inner:]
    hq, hs = _quantize(g / (1.0 + torch.exp(-g)) * u)
    if T * k < E:
        picked = torch.matmul(w_down, hq[..., None])[..., 0] * hs * s_down       # (T, k, H)
    else:
        down = torch.matmul(hq, s["w_down"].float().transpose(1, 2)) * hs * s["s_down"][:, None, :]
        picked = down.transpose(0, 1)[torch.arange(T, device=x.device)[:, None], ids]
    y = (picked * gates[..., None]).sum(1)
    return {"y": y.to(s["x"].dtype), "ids": ids.to(torch.int32), "gates": gates}


def run(s):
    case = s["case"]
    if not own:
        return {"rows": _plain_rows, "linear": _plain_linear, "moe": _plain_moe}[case["op"]](s)
    import dense_fp32_matrix_row_gb300 as sg
    if case["op"] == "rows":
        if case["norm"]:
            sg.rmsnorm_q8(s["x"], s["weight"], s["q"], s["scale"], residual=s["residual"], h=s["h"],
                          y=s["y"], eps=1e-6)
        else:
            sg.quantize_q8(s["x"], s["q"], s["scale"])
        out = {"q": s["q"], "scale": s["scale"]}
        out.update({n: s[n] for n in ("h", "y") if s[n] is not None})
        return out
    if case["op"] == "linear":
        sg.linear_q8(s["xq"], s["xs"], s["wq"], s["ws"], s["out"], bias=s["bias"],
                     activation=case["act"])
        return s["out"]
    sg.moe_q8(s["x"], s["router"], s["w_up"], s["s_up"], s["w_down"], s["s_down"], s["out"],
              top_k=case["k"], renormalize=case["renorm"], ids=s["ids"], gates=s["gates"])
    return {"y": s["out"], "ids": s["ids"], "gates": s["gates"]}


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rows":
        M, K = case["M"], case["K"]
        per = size * (1 + 2 * case["residual"] + case["y"]) + 1
        return {"bytes": M * K * per + 4 * M + (4 * K if case["norm"] else 0), "flops": 6 * M * K}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + size * M * N + 4 * (M + N), "flops": 2 * M * N * K}
    T, E, k, H, inner = (case[n] for n in ("T", "E", "k", "H", "I"))
    # experts that some token picks, on average
    touched = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": touched * (3 * H * inner + 4 * (2 * inner + H)) + 4 * E * H + 2 * size * T * H,
            "flops": 2 * T * E * H + 6 * T * k * H * inner}


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "rows":
        h = s["x"].to(d)
        out = {"q": None}
        if s["residual"] is not None:
            h = h + s["residual"].to(d)
            out["h"] = h
        rms = 1.0
        w = 1.0
        if case["norm"]:
            rms = ((h ** 2).sum(1, keepdim=True) / case["K"] + 1e-6) ** 0.5
            w = s["weight"].to(d)
        normed = h / rms * w
        if case["y"]:
            out["y"] = normed
        out["scale"] = normed.abs().max(1).values / 127
        return out
    if case["op"] == "linear":
        if case["M"] * case["N"] * case["K"] > 8192 * 14336 * 4096:
            return None
        out = torch.empty((case["M"], case["N"]), dtype=d, device="cuda")
        wt = s["wq"].to(d).t().contiguous()
        for m0 in range(0, case["M"], 1024):
            rows = slice(m0, min(m0 + 1024, case["M"]))
            c = torch.einsum("mk,kn->mn", s["xq"][rows].to(d), wt)
            c *= s["xs"][rows].to(d).unsqueeze(1)
            c *= s["ws"].to(d)
            if s["bias"] is not None:
                c += s["bias"].to(d)
            if case["act"] == "relu":
                c = c.clamp(min=0)
            elif case["act"] == "gelu":
                c = c * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (c + 0.044715 * c ** 3))
            elif case["act"] == "silu":
                c = c * torch.sigmoid(c)
            out[rows] = c
        return out
    T, k, inner = case["T"], case["k"], case["I"]
    x = s["x"].to(d)
    out = torch.zeros((T, case["H"]), dtype=d, device="cuda")
    gates = torch.zeros((T, k), dtype=d, device="cuda")
    for t in range(T):
        logits = (s["router"].to(d) * x[t]).sum(1)
        e = torch.exp(logits - logits.max())
        order = sorted(range(case["E"]), key=lambda i: (-float(e[i]), i))[:k]
        weight = e[order] / (e[order].sum() if case["renorm"] else e.sum())
        gates[t] = weight
        step = x[t].abs().max() / 127
        xq = torch.round(x[t] / step)
        for j, i in enumerate(order):
            up = (s["w_up"][i].to(d) @ xq) * step * s["s_up"][i].to(d)
            hid = up[:inner] * torch.sigmoid(up[:inner]) * up[inner:]
            hstep = hid.abs().max() / 127
            out[t] += weight[j] * (s["w_down"][i].to(d) @ torch.round(hid / hstep)) * hstep * s["s_down"][i].to(d)
    return {"y": out, "ids": None, "gates": gates}
