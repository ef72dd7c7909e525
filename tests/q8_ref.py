"""64-bit restatements of the 8-bit operators, and padded device arrays, for
their tests.

The whole numbers of a quantised row are defined by FP32 operations (one
product, one division, one product, one rounding), which numpy's float32 does
bit for bit; everything else is float64.
"""

from __future__ import annotations

import math

import numpy as np

F32 = np.float32


def quantize(p):
    """(q int64, step float64) of each row of the float32 array `p`."""
    p = np.asarray(p, dtype=F32)
    q = np.zeros(p.shape, dtype=np.int64)
    step = np.zeros(p.shape[0])
    for r in range(p.shape[0]):
        row = p[r]
        if row.size == 0:
            continue
        if not np.isfinite(row).all():
            step[r] = np.nan
            continue
        m = np.abs(row).max()
        if m == 0:
            continue
        lift = F32(2.0 ** 100) if m < F32(2.0 ** -100) else F32(1)
        q[r] = np.rint((row * lift) * (F32(127) / (m * lift))).astype(np.int64)
        step[r] = float(m) / 127.0
    return q, step


def bf16_round(x):
    """float64 -> the nearest bf16 (ties to even) as float64, through float32
    (exact enough for values that are float32 already)."""
    b = np.asarray(x, dtype=F32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(F32).astype(np.float64)


def activation(v, act):
    v = np.asarray(v, dtype=np.float64)
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    if act == "gelu":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    return v


def linear(xq, xs, wq, ws, bias, act):
    """(result, size): the result in float64, and |product| + |bias| of each
    element, which its FP32 roundings are relative to."""
    # exact: |sum| <= 131071 * 2^14 < 2^53
    v = (xq.astype(np.float64) @ wq.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None]
    size = np.abs(v)
    if bias is not None:
        v = v + bias.astype(np.float64)[None]
        size = size + np.abs(bias.astype(np.float64))[None]
    return activation(v, act), size


def moe(x, router, w_up, s_up, w_down, s_down, k, renorm):
    """(out, slack, ids, gates, gap) of the expert layer.

    `slack` bounds what a hidden value that lies within 2e-4 of a rounding
    boundary can move the result by: such a value may round either way, since
    hid carries a few FP32 roundings and expf's error (about 1e-6 relative, so
    127e-6 of a step).  `gap` is the smallest difference between a chosen
    logit and the next."""
    T, H = x.shape
    E, inner = s_down.shape[0], w_down.shape[2]
    x64 = x.astype(np.float64)
    logits = x64 @ router.astype(np.float64).T
    xq, xstep = quantize(x)
    out, slack = np.zeros((T, H)), np.zeros((T, H))
    ids, gates = np.zeros((T, k), dtype=np.int64), np.zeros((T, k))
    gap = np.inf
    for t in range(T):
        order = np.lexsort((np.arange(E), -logits[t]))
        ids[t] = order[:k]
        srt = logits[t][order[:min(k + 1, E)]]
        if len(srt) > 1:
            gap = min(gap, float(np.min(-np.diff(srt))))
        e = np.exp(logits[t] - logits[t].max())
        gates[t] = e[ids[t]] / (e[ids[t]].sum() if renorm else e.sum())
        for j in range(k):
            i = ids[t, j]
            up = (w_up[i].astype(np.float64) @ xq[t]) * xstep[t] * s_up[i].astype(np.float64)
            hid = activation(up[:inner], "silu") * up[inner:]
            step = np.abs(hid).max() / 127.0
            n = hid / step if step > 0 else np.zeros(inner)
            hq = np.rint(n)
            unsure = np.abs(np.abs(n - np.trunc(n)) - 0.5) < 2e-4
            scale = gates[t, j] * step * s_down[i].astype(np.float64)
            out[t] += (w_down[i].astype(np.float64) @ hq) * scale
            slack[t] += (np.abs(w_down[i].astype(np.float64)) @ unsure) * np.abs(scale)
            # each expert's own terms, whose FP32 roundings a sum of them keeps
            slack[t] += 2.0 ** -19 * np.abs((w_down[i].astype(np.float64) @ hq) * scale)
            # the scale of the hidden row moves with its maximum, 1e-6 relative
            slack[t] += 2e-6 * np.abs((w_down[i].astype(np.float64) @ hq) * scale)
    return out, slack, ids, gates, gap


class Padded:
    """A rows x cols device array of any element type with row stride `ld`,
    `offset` elements into its buffer, and a byte pattern all around it."""

    FILL = 0xA5

    def __init__(self, X, ld=None, offset=0, guard=64):
        import torch
        self.t = X if isinstance(X, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(X))
        rows, cols = self.t.shape
        ld = max(cols, 1) if ld is None else ld
        n = guard + offset + rows * ld + guard
        size = self.t.element_size()
        self.buf = torch.full((n * size,), self.FILL, dtype=torch.uint8, device="cuda")
        typed = self.buf.view(self.t.dtype)
        self.view = torch.as_strided(typed, (rows, cols), (ld, 1), guard + offset)
        self.view.copy_(self.t)
        mask = torch.zeros(n, dtype=torch.bool, device="cuda")
        if rows and cols:
            torch.as_strided(mask, (rows, cols), (ld, 1), guard + offset).fill_(True)
        self.inside = mask.repeat_interleave(size)
        self.before = self.buf.clone()

    def outside_intact(self):
        return bool((self.buf[~self.inside] == self.FILL).all())

    def unchanged(self):
        return bool((self.buf == self.before).all())
