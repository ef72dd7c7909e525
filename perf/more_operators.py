"""Workloads of the attention operators that serve from an 8-bit key-value cache:
norms of queries and keys with the position rotation, the cache's write and read,
and attention of one new token per sequence over the cache's pages.

``run`` computes each in plain 32-bit torch operations, or, where ``own`` is
true, through the package's entry points.  ``exact`` restates the definitions
in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one decoded token's heads: the launch is all there is
        {"name": "rope_token", "op": "rope", "T": 1, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "dtype": "bf16",
         "norm": True, "interleaved": False, "start": 100000},
        # a prompt's heads, taken from the rows of a joint projection
        {"name": "rope_prompt", "op": "rope", "T": 8192, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "dtype": "bf16",
         "norm": True, "interleaved": False, "start": 0},
        # heads that are no power of two, a part of each rotated, neighbours paired, no norm
        {"name": "rope_part_fp32", "op": "rope", "T": 1001, "Hq": 14, "Hk": 2, "D": 80, "R": 32, "dtype": "fp32",
         "norm": False, "interleaved": True, "start": 5000},
        # sixteen decoded sequences' new tokens into the cache, and read back
        {"name": "cache_decode_16", "op": "cache", "T": 16, "N": 16, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "page": 16, "dtype": "bf16", "rope": True, "norm": True, "interleaved": False, "start": 4096},
        # a chunk of a long prompt: its tokens are written, it and all before it read for the chunk's attention
        {"name": "cache_chunk", "op": "cache", "T": 2048, "N": 18432, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "page": 16, "dtype": "bf16", "rope": True, "norm": True, "interleaved": False, "start": 16384},
        # keys that are rotated already, short heads, large pages
        {"name": "cache_rotated_64", "op": "cache", "T": 8192, "N": 8192, "Hq": 0, "Hk": 8, "D": 64, "R": 0,
         "page": 64, "dtype": "bf16", "rope": False, "norm": False, "interleaved": False, "start": 0},
        # FP32 rows, odd counts, pages that are no power of two
        {"name": "cache_odd_fp32", "op": "cache", "T": 777, "N": 1001, "Hq": 10, "Hk": 5, "D": 96, "R": 64,
         "page": 20, "dtype": "fp32", "rope": True, "norm": True, "interleaved": False, "start": 333},
        # one chat with a short history: latency
        {"name": "attend_token", "op": "attend", "B": 1, "L": 500, "Hk": 8, "G": 4, "D": 128, "page": 16,
         "dtype": "bf16", "window": 0, "ragged": False},
        # one sequence with a long history: the cache is divided over the GPU
        {"name": "attend_long", "op": "attend", "B": 1, "L": 131072, "Hk": 8, "G": 4, "D": 128, "page": 16,
         "dtype": "bf16", "window": 0, "ragged": False},
        # a decode batch of unequal lengths, some slots of the batch unused
        {"name": "attend_batch", "op": "attend", "B": 64, "L": 8192, "Hk": 8, "G": 8, "D": 128, "page": 16,
         "dtype": "bf16", "window": 0, "ragged": True},
        # the largest batch of long sequences
        {"name": "attend_large", "op": "attend", "B": 64, "L": 16384, "Hk": 8, "G": 8, "D": 128, "page": 32,
         "dtype": "bf16", "window": 0, "ragged": False},
        # FP32, odd head counts and sizes, pages that end inside a tile, a sliding window
        {"name": "attend_odd_fp32", "op": "attend", "B": 7, "L": 3001, "Hk": 3, "G": 5, "D": 80, "page": 20,
         "dtype": "fp32", "window": 1000, "ragged": True},
    ]


def _size(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "cache", "attend", "attend"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    D = rng.choice((64, 64, 80, 96, 112, 128, 128, 128, 192, 256))
    page = rng.choice((16, 16, 32, 64, 128, 8, 20))
    if op == "attend":
        Hk, G = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 2, 4, 5, 7, 8, 12, 16, 24))
        B = _size(rng, 1, 256)
        most = (64 * 16384 * 8 * 128 * 8) // (B * Hk * D * max(8, G))     # the largest listed case's work
        L = _size(rng, 16, max(17, min(131072, most)))
        return {"op": op, "B": B, "L": L, "Hk": Hk, "G": G, "D": D, "page": page, "dtype": dtype,
                "window": _size(rng, 1, L) if rng.random() < 0.25 else 0, "ragged": rng.random() < 0.7}
    Hk = rng.choice((1, 2, 4, 5, 8))
    Hq = Hk * rng.choice((1, 2, 4, 5, 8))
    T = _size(rng, 1, min(8192, (8192 * 40 * 128) // ((Hq + Hk) * D)))
    rope = op == "rope" or rng.random() < 0.7
    R = rng.choice((D, D, D // 2, 32)) if rope else 0
    case = {"op": op, "T": T, "Hq": Hq if rope else 0, "Hk": Hk, "D": D, "R": R, "dtype": dtype,
            "norm": rope and rng.random() < 0.6, "interleaved": rope and rng.random() < 0.3,
            "start": _size(rng, 1, 100000)}
    if op == "cache":
        case.update(N=T + (_size(rng, 1, 8192) if rng.random() < 0.5 else 0), page=page, rope=rope)
    return case


def _lens(case):
    """Tokens of each sequence: all L, or spread over [L/8, L] with every ninth slot unused."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    r = random.Random(B * 1000003 + L)
    return [0 if b % 9 == 8 else L if b == 0 else r.randint(max(1, L // 8), L) for b in range(B)]


def _int8(gen, *shape):
    """8-bit values as a row of normal numbers gives them: a deviation of about 32."""
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return v.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(gen, *shape):
    return (0.5 + torch.rand(shape, generator=gen, device="cuda")) / 32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, D, Hk = DTYPES[case["dtype"]], case["D"], case["Hk"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] == "attend":
        B, L, page = case["B"], case["L"], case["page"]
        lens = _lens(case)
        pages = [-(-n // page) for n in lens]
        width = max(1, -(-L // page))
        blocks = sum(pages) + 3
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        # each sequence's pages lie anywhere in the pool; entries behind them are -1
        count = torch.tensor(pages, device="cuda")
        at = (torch.cumsum(count, 0) - count)[:, None] + torch.arange(width, device="cuda")
        used = torch.arange(width, device="cuda") < count[:, None]
        s["table"] = torch.where(used, order[torch.where(used, at, 0)], -1).to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["q"] = (2.0 * normal(B, Hk * case["G"], D)).to(dt)
        s["k"], s["k_scale"] = _int8(gen, blocks, Hk, page, D), _scales(gen, blocks, Hk, page)
        s["v"], s["v_scale"] = _int8(gen, blocks, Hk, page, D), _scales(gen, blocks, Hk, page)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hk * case["G"]), device="cuda")
    else:
        T, Hq, R = case["T"], case["Hq"], case["R"]
        # the rows of a joint projection: queries, keys and values side by side
        rows = normal(T, Hq + 2 * Hk, D)
        rows[:, :, :: max(1, D // 5)] *= 4.0
        rows = rows.to(dt)
        s["q"], s["k_new"], s["v_new"] = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
        if R:
            count = case["start"] + T
            angle = torch.arange(count, device="cuda", dtype=torch.float64)[:, None] * (
                10000.0 ** (-2.0 * torch.arange(R // 2, device="cuda", dtype=torch.float64) / R))
            s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
            s["positions"] = torch.arange(case["start"], count, device="cuda")
            s["q_out"] = torch.empty((T, Hq, D), device="cuda", dtype=dt)
        s["q_weight"] = 1.0 + 0.2 * normal(D) if case["norm"] else None
        s["k_weight"] = 1.0 + 0.2 * normal(D) if case["norm"] else None
        if case["op"] == "rope":
            s["k_out"] = torch.empty((T, Hk, D), device="cuda", dtype=dt)
        else:
            N, page = case["N"], case["page"]
            blocks = -(-N // page) + 3
            order = torch.randperm(blocks, generator=gen, device="cuda")
            t = torch.arange(N, device="cuda")
            s["read"] = order[t // page] * page + t % page       # the sequence's tokens, page by page
            s["slots"] = s["read"][N - T:].clone()               # the new ones are its last
            s["k"], s["k_scale"] = _int8(gen, blocks, Hk, page, D), _scales(gen, blocks, Hk, page)
            s["v"], s["v_scale"] = _int8(gen, blocks, Hk, page, D), _scales(gen, blocks, Hk, page)
            s["k_out"] = torch.empty((N, Hk, D), device="cuda", dtype=dt)
            s["v_out"] = torch.empty((N, Hk, D), device="cuda", dtype=dt)
    return s


def _rotate(p, cos, sin, interleaved):
    """The first R channels of each head rotated in pairs; cos and sin are (T, R/2)."""
    half = cos.shape[1]
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = p[..., 0:2 * half:2], p[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = p[..., :half], p[..., half:2 * half]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, p[..., 2 * half:]), -1)


def _plain_heads(s, x, weight):
    """(p, r): the heads are p * r, r the norm's factor of each (1 without a norm)."""
    x = x.float()
    p, r = x, torch.ones_like(x[..., :1])
    if weight is not None:
        p, r = x * weight, 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    if s["case"]["R"]:
        at = s["positions"]
        p = _rotate(p, s["cos"][at], s["sin"][at], s["case"]["interleaved"])
    return p, r


def _quantize(p):
    """Whole numbers rint(p * 127/max|p|) of each row, and the row's max|p| / 127."""
    m = p.abs().amax(-1, keepdim=True)
    top = torch.full_like(m, 127.0)      # a tensor: dividing by or into a number multiplies by a reciprocal
    q = torch.where(m > 0, torch.round(p * (top / m)), torch.zeros_like(p))
    return q.to(torch.int8), m / top


def _plain_rope(s):
    out = {}
    for name, x, w in (("q", s["q"], s["q_weight"]), ("k", s["k_new"], s["k_weight"])):
        p, r = _plain_heads(s, x, w)
        out[name] = (p * r).to(x.dtype)
    return out


def _plain_cache(s):
    case, out = s["case"], {}
    dt = s["k_new"].dtype
    if case["rope"]:
        p, r = _plain_heads(s, s["q"], s["q_weight"])
        out["q"] = (p * r).to(dt)
    page = case["page"]
    block, row = s["slots"] // page, s["slots"] % page
    p, r = _plain_heads(s, s["k_new"], s["k_weight"])
    q, step = _quantize(p)
    s["k"][block, :, row], s["k_scale"][block, :, row] = q, (step * r)[..., 0]
    q, step = _quantize(s["v_new"].float())
    s["v"][block, :, row], s["v_scale"][block, :, row] = q, step[..., 0]
    block, row = s["read"] // page, s["read"] % page
    for name in ("k", "v"):
        out[name] = (s[name][block, :, row].float() * s[name + "_scale"][block, :, row][..., None]).to(dt)
    return out


def _plain_attend(s):
    case = s["case"]
    B, Hk, G, D, page = (case[n] for n in ("B", "Hk", "G", "D", "page"))
    table, lens = s["table"].clamp(min=0).long(), s["lens"]
    width = table.shape[1]

    def rows(name):
        x = s[name][table].float() * s[name + "_scale"][table][..., None]        # (B, width, Hk, page, D)
        return x.transpose(1, 2).reshape(B, Hk, width * page, D)

    q = s["q"].float().view(B, Hk, G, D)
    scores = torch.matmul(q, rows("k").transpose(-1, -2)) * (1.0 / math.sqrt(D))  # (B, Hk, G, width * page)
    t = torch.arange(width * page, device=q.device)
    seen = t < lens[:, None]
    if case["window"]:
        seen = seen & (t >= lens[:, None] - case["window"])
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    # what no sequence holds is not read: a masked value counts as 0, whatever it is
    v = torch.where(seen[:, None, :, None], rows("v"), 0.0)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return {"out": out.reshape(B, Hk * G, D).to(s["q"].dtype), "lse": (m + torch.log(total)).reshape(B, Hk * G)}


def run(s):
    case = s["case"]
    if not own:
        return {"rope": _plain_rope, "cache": _plain_cache, "attend": _plain_attend}[case["op"]](s)
    import dense_fp32_matrix_row_gb300 as sg
    if case["op"] == "rope":
        sg.norm_rope(s["q"], s["k_new"], s["cos"], s["sin"], s["q_out"], s["k_out"], positions=s["positions"],
                     q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if "cache" not in s:        # a program wraps its pool once
        s["cache"] = sg.CacheQ8(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "cache":
        out = {"k": s["k_out"], "v": s["v_out"]}
        if case["rope"]:
            sg.norm_rope_write_q8(s["q"], s["k_new"], s["v_new"], s["cos"], s["sin"], s["q_out"], s["cache"],
                                  s["slots"], positions=s["positions"], q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"])
            out["q"] = s["q_out"]
        else:
            sg.cache_write_q8(s["k_new"], s["v_new"], s["cache"], s["slots"])
        sg.cache_read_q8(s["cache"], s["read"], s["k_out"], s["v_out"])
        return out
    sg.attend_q8(s["q"], s["cache"], s["table"], s["lens"], s["out"], window=case["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    D, Hk = case["D"], case["Hk"]
    if case["op"] == "attend":
        lens = [min(n, case["window"]) if case["window"] else n for n in _lens(case)]
        rows = sum(lens) * Hk
        heads = case["B"] * Hk * case["G"]
        return {"bytes": 2 * rows * (D + 4) + heads * (2 * D * size + 4) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 4 * rows * case["G"] * D}
    T, Hq, R = case["T"], case["Hq"], case["R"]
    table = 4 * T * R + (8 * T if R else 0)
    if case["op"] == "rope":
        return {"bytes": 2 * T * (Hq + Hk) * D * size + table, "flops": 8 * T * (Hq + Hk) * D}
    N = case["N"]
    return {"bytes": T * (2 * Hq + 2 * Hk) * D * size + table + 2 * T * Hk * (D + 4) + 8 * T
            + 2 * N * Hk * (D + 4 + D * size) + 8 * N,
            "flops": 8 * T * (Hq + 2 * Hk) * D + 2 * N * Hk * D}


def _exact_heads(s, x, weight):
    d, R = torch.float64, s["case"]["R"]
    x = x.to(d)
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) ** 0.5 * weight.to(d)
    if not R:
        return x
    # each pair as a complex number, turned by its angle
    turn = torch.complex(s["cos"].to(d), s["sin"].to(d)).index_select(0, s["positions"]).unsqueeze(1)
    head = x[..., :R].unflatten(-1, (R // 2, 2) if s["case"]["interleaved"] else (2, R // 2))
    if not s["case"]["interleaved"]:
        head = head.transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    if not s["case"]["interleaved"]:
        turned = turned.transpose(-1, -2)
    x = x.clone()
    x[..., :R] = turned.flatten(-2)
    return x


def _exact_values(x):
    """What the nearest 127ths of each row's largest magnitude stand for."""
    step = x.abs().max(-1, keepdim=True).values / 127
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "rope":
        return {"q": _exact_heads(s, s["q"], s["q_weight"]), "k": _exact_heads(s, s["k_new"], s["k_weight"])}
    if case["op"] == "cache":
        out = {"q": _exact_heads(s, s["q"], s["q_weight"])} if case["rope"] else {}
        if case["dtype"] == "fp32":
            # a value next to a border between two 8-bit numbers may go either way: 1/127 where the type keeps 1e-7
            return {**out, "k": None, "v": None} if out else None
        N, T, page = case["N"], case["T"], case["page"]
        fresh = {"k": _exact_heads(s, s["k_new"], s["k_weight"]), "v": s["v_new"].to(d)}
        for name, x in fresh.items():
            pool = (s[name].to(d) * s[name + "_scale"].to(d).unsqueeze(-1)).transpose(1, 2).flatten(0, 1)
            pool.index_copy_(0, s["slots"], _exact_values(x))
            out[name] = pool.index_select(0, s["read"])
        return out
    B, Hk, G, D, page = (case[n] for n in ("B", "Hk", "G", "D", "page"))
    out = torch.zeros((B, Hk * G, D), device="cuda", dtype=d)
    lse = torch.full((B, Hk * G), -math.inf, device="cuda", dtype=d)
    for b, n in enumerate(_lens(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        t = torch.arange(first, n, device="cuda")
        block, row = s["table"][b].long()[t // page], t % page
        k = s["k"][block, :, row].to(d) * s["k_scale"][block, :, row].to(d).unsqueeze(-1)       # (n, Hk, D)
        v = s["v"][block, :, row].to(d) * s["v_scale"][block, :, row].to(d).unsqueeze(-1)
        q = s["q"][b].to(d).unflatten(0, (Hk, G))
        logits = torch.einsum("hgd,nhd->hgn", q, k) / D ** 0.5
        out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(logits, -1), v).flatten(0, 1)
        lse[b] = torch.logsumexp(logits, -1).flatten()
    return {"out": out, "lse": lse}
