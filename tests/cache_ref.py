"""64-bit restatements of the attention operators over the 8-bit cache, with bounds
of what FP32 arithmetic may add, and random pools for their tests.

The whole numbers of a quantised row are defined by FP32 operations (products,
sums and differences of pairs, each rounded by itself), which numpy's float32
does bit for bit; everything else is float64.
"""

from __future__ import annotations

import numpy as np
import torch

import q8_ref

F32 = np.float32


def pairs(D, R, interleaved):
    """Index arrays (a, b) of the R/2 rotated pairs."""
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate32(p, cos, sin, interleaved):
    """p (T, H, D) float32 with its pairs turned; cos, sin (T, R/2) float32."""
    a, b = pairs(p.shape[-1], 2 * cos.shape[1], interleaved)
    c, s = cos[:, None], sin[:, None]
    out = p.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        out[..., a] = p[..., a] * c - p[..., b] * s
        out[..., b] = p[..., b] * c + p[..., a] * s
    return out


def norm_rope(x, weight, cos, sin, interleaved, eps):
    """(p32, r, y, size) of heads x (T, H, D) float32: FP32's own p, the norm's factor
    and the result in 64 bits, and the size that its FP32 roundings are relative to."""
    x64 = x.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        p32 = x if weight is None else x * weight
    p64 = x64 if weight is None else x64 * weight.astype(np.float64)
    size = np.abs(p64)
    if cos is not None:
        p32 = rotate32(p32, cos, sin, interleaved)
        a, b = pairs(x.shape[-1], 2 * cos.shape[1], interleaved)
        c, s = cos.astype(np.float64)[:, None], sin.astype(np.float64)[:, None]
        turned, big = p64.copy(), size.copy()
        with np.errstate(invalid="ignore"):
            turned[..., a] = p64[..., a] * c - p64[..., b] * s
            turned[..., b] = p64[..., b] * c + p64[..., a] * s
            big[..., a] = np.abs(p64[..., a] * c) + np.abs(p64[..., b] * s)
            big[..., b] = np.abs(p64[..., b] * c) + np.abs(p64[..., a] * s)
        p64, size = turned, big
    r = np.ones(x.shape[:2])
    if weight is not None:
        with np.errstate(invalid="ignore", divide="ignore"):
            r = 1.0 / np.sqrt((x64 ** 2).mean(-1) + eps)
    with np.errstate(invalid="ignore"):
        return p32, r, p64 * r[..., None], size * np.abs(r)[..., None]


def quantize(p32, r):
    """(q, scale) of heads p32 (T, H, D) whose norm's factor is r (T, H)."""
    q, step = q8_ref.quantize(p32.reshape(-1, p32.shape[-1]))
    with np.errstate(invalid="ignore"):
        scale = np.where(step == 0, 0.0, step * r.reshape(-1))
    return q.reshape(p32.shape), scale.reshape(p32.shape[:2])


class Pool:
    """Random pages on the GPU.  What no token lies in holds whole numbers of any
    size and NaN scales."""

    def __init__(self, blocks, heads, page, dim, seed=0, scale=1 / 32, pad=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.blocks, self.heads, self.page, self.dim = blocks, heads, page, dim
        rows = heads * page

        def pages(each, dtype, extra):      # pages `extra` elements apart
            return torch.empty((blocks, each + extra), device="cuda", dtype=dtype)[:, :each]

        self.k, self.v = (pages(rows * dim, torch.int8, 16 * pad).view(blocks, heads, page, dim) for _ in range(2))
        self.k_scale, self.v_scale = (pages(rows, torch.float32, 3 * pad).view(blocks, heads, page) for _ in range(2))
        for t in (self.k, self.v):
            t.copy_(torch.randint(-127, 128, t.shape, generator=gen, device="cuda", dtype=torch.int8))
        for t in (self.k_scale, self.v_scale):
            t.copy_((0.25 + torch.rand(t.shape, generator=gen, device="cuda")) * scale / 2)

    def cache(self):
        import dense_fp32_matrix_row_gb300 as sg
        return sg.CacheQ8(self.k, self.v, self.k_scale, self.v_scale)

    def table(self, lens, width=None, seed=0):
        """(table, kept): pages in random order for sequences of these lengths, and a
        mask (blocks, page) of the rows that some token lies in.  Unused entries
        of the table name pages outside the pool."""
        need = [-(-n // self.page) for n in lens]
        width = max([1] + need) if width is None else width
        order = np.random.default_rng(seed).permutation(self.blocks)
        table = np.full((len(lens), width), self.blocks + 7, dtype=np.int32)
        kept = np.zeros((self.blocks, self.page), dtype=bool)
        at = 0
        for b, n in enumerate(lens):
            own = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = own
            for i, page in enumerate(own):
                kept[page, :min(self.page, n - i * self.page)] = True
        assert at <= self.blocks
        return torch.from_numpy(table).cuda(), torch.from_numpy(kept).cuda()

    def poison(self, kept):
        """NaN scales and the number -128 in every row that is not kept."""
        off = ~kept[:, None].expand(self.blocks, self.heads, self.page)
        for t in (self.k, self.v):
            t.masked_fill_(off[..., None], -128)
        for t in (self.k_scale, self.v_scale):
            t.masked_fill_(off, float("nan"))


def attend(q, pool, table, lens, scale, window, bf16, drop=None):
    """(out, tol, lse, lse_tol) in 64 bits (on the GPU), tol without the output type's
    rounding.

    Bounds, in units of u = 2^-23 (twice FP32's half step: an MMA may cut what it adds).
    A score: the query's second FP16 term leaves 2^-22 of each element, D/16 MMAs (twice with two
    terms) add to a running sum below size = scale * sum |q_d k_d|, and five factors and
    the difference to m are rounded: s moves by (2 + D/8 + 8) u of size (|s| <= size).  p:
    that, and exp2's two units and the factors' three: 6 u.  A sum over n tokens: at most
    n/16 + 24 additions.  The probabilities' rounding to FP16: 2^-11 (2^-22 with two terms).
    Numerator and denominator each carry p's error.

    FP16's smallest step is 2^-24.  The products p * (value scale) are held as multiples of
    a power of two that takes the largest value scale to 2^8 or more (the scale that sets it
    is one of the sequence's, taken to [2^8, 2^9)), at p = 1 for a score that is no larger
    than the sequence's largest.  Each is off by at most half a step, 2^-25 there, so 2^-33 of
    the largest value scale once the sum of p (at least 1 then) divides it, times a whole
    number of up to 127; exp2's results below 2^-126, taken as 0, are less."""
    B, H, D = q.shape
    Hk, page = pool.heads, pool.page
    G, u = H // Hk, 2.0 ** -23
    d = torch.float64
    out, tol = torch.zeros((B, H, D), dtype=d, device="cuda"), torch.zeros((B, H, D), dtype=d, device="cuda")
    lse = torch.full((B, H), float("-inf"), dtype=d, device="cuda")
    lse_tol = torch.zeros((B, H), dtype=d, device="cuda")
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * page))
        first = max(0, n - window) if window else 0
        t = torch.arange(first, n, device="cuda")
        block, row = table[b].long()[t // page], t % page
        fine = (block >= 0) & (block < pool.blocks)
        block, row = block[fine], row[fine]
        if len(block) == 0:
            continue
        k = pool.k[block, :, row].to(d) * pool.k_scale[block, :, row].to(d)[..., None]      # (n, Hk, D)
        v = pool.v[block, :, row].to(d) * pool.v_scale[block, :, row].to(d)[..., None]
        x = q[b].to(d).view(Hk, G, D)
        s = torch.einsum("hgd,nhd->hgn", x, k) * scale
        size = torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()) * abs(scale)
        p = torch.softmax(s, -1)
        out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(H, D)
        lse[b] = torch.logsumexp(s, -1).reshape(H)
        eps = (10 + D / 8) * u * size.amax(-1) + 6 * u
        adds = (n / 16 + 24) * u
        weight = torch.einsum("hgn,nhd->hgd", p, v.abs())
        least = 127 * len(block) * 2.0 ** -33 * pool.v_scale[block, :, row].to(d).abs().amax(0)      # (Hk)
        tol[b] = (weight * (2 * eps + 2 * adds + (2.0 ** -11 if bf16 else 2.0 ** -21))[..., None]
                  + least[:, None, None]).reshape(H, D)
        lse_tol[b] = (eps + adds + 4 * u * (1 + lse[b].view(Hk, G).abs())).reshape(H)
    return out, tol, lse, lse_tol
