"""A feed-forward block served in 8 bits, dense and with experts.

The chain a decoder layer runs behind its attention, with every product in 8-bit
whole numbers and the residual stream in bfloat16:

    h, q   = residual addition, RMS norm and quantisation     (rmsnorm_q8)
    hidden = SiLU(q @ W_up^T)                                 (linear_q8)
    qh     = the hidden rows in 8 bits                        (quantize_q8)
    out    = qh @ W_down^T                                    (linear_q8)

or, for up to 64 tokens, the same position taken by a mixture of experts that
reads the normalised rows:

    out    = experts(y)                                       (moe_q8)

``out`` is the residual of the next block's norm.  Weights are quantised once,
one scale per output channel, with the same quantize_q8.

    python examples/q8_feed_forward.py                # a decode batch, dense and experts
    python examples/q8_feed_forward.py --tokens 2048  # a prompt, dense

prints the time of a block and its distance from the same block in FP32 (the
library's own FP32 product on the unquantised weights).
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_row_gb300 as sg  # noqa: E402


def quantized(w):
    """(N, K) weights as (8-bit rows, scales), any number of leading experts."""
    rows = w.reshape(-1, w.shape[-1])
    q = torch.empty(rows.shape, dtype=torch.int8, device=w.device)
    s = torch.empty(rows.shape[0], device=w.device)
    sg.quantize_q8(rows, q, s)
    return q.view(w.shape), s.view(w.shape[:-1])


class Norm:
    """Residual addition and RMS norm into 8-bit rows, with buffers for `tokens` rows."""

    def __init__(self, weight, tokens, eps=1e-6):
        hidden = weight.numel()
        self.weight, self.eps = weight, eps
        self.q = torch.empty((tokens, hidden), dtype=torch.int8, device=weight.device)
        self.scale = torch.empty(tokens, device=weight.device)
        self.y = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=weight.device)

    def __call__(self, x, stream_rows, want_y=False):
        """stream_rows += x in place; the norm of the sum stays in q, scale (and y)."""
        sg.rmsnorm_q8(x, self.weight, self.q, self.scale, residual=stream_rows, h=stream_rows,
                      y=self.y if want_y else None, eps=self.eps)


class DenseBlock:
    def __init__(self, norm, w_up, w_down):
        self.norm = norm
        (self.w_up, self.s_up), (self.w_down, self.s_down) = quantized(w_up), quantized(w_down)
        tokens, dev = norm.q.shape[0], w_up.device
        inner, hidden = w_up.shape
        self.hidden = torch.empty((tokens, inner), dtype=torch.bfloat16, device=dev)
        self.hq = torch.empty((tokens, inner), dtype=torch.int8, device=dev)
        self.hs = torch.empty(tokens, device=dev)
        self.out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=dev)

    def __call__(self, x, stream_rows):
        n = self.norm
        n(x, stream_rows)
        sg.linear_q8(n.q, n.scale, self.w_up, self.s_up, self.hidden, activation="silu")
        sg.quantize_q8(self.hidden, self.hq, self.hs)
        sg.linear_q8(self.hq, self.hs, self.w_down, self.s_down, self.out)
        return self.out


class ExpertBlock:
    def __init__(self, norm, router, w_up, w_down, top_k):
        self.norm, self.router, self.top_k = norm, router, top_k
        (self.w_up, self.s_up), (self.w_down, self.s_down) = quantized(w_up), quantized(w_down)
        self.out = torch.empty_like(norm.y)

    def __call__(self, x, stream_rows):
        self.norm(x, stream_rows, want_y=True)
        sg.moe_q8(self.norm.y, self.router, self.w_up, self.s_up, self.w_down, self.s_down, self.out, self.top_k)
        return self.out


def fp32_product(a, w):
    """a @ w^T by the library's FP32 product."""
    c = torch.empty((a.shape[0], w.shape[0]), device=a.device)
    sg.sgemm(a.contiguous(), w.t().contiguous(), c)
    return c


def silu(v):
    return v / (1 + torch.exp(-v))


def fp32_norm(x, stream_rows, weight, eps=1e-6):
    h = x.float() + stream_rows.float()
    return h * weight / torch.sqrt((h * h).mean(1, keepdim=True) + eps)


def fp32_dense(y, w_up, w_down):
    return fp32_product(silu(fp32_product(y, w_up)), w_down)


def fp32_experts(y, router, w_up, w_down, top_k):
    logits = fp32_product(y, router)
    top, ids = torch.topk(logits, top_k)
    gates = torch.exp(top - top[:, :1])
    gates = gates / gates.sum(1, keepdim=True)
    inner = w_down.shape[2]
    out = torch.zeros_like(y)
    for t in range(y.shape[0]):
        for j in range(top_k):
            e = int(ids[t, j])
            up = fp32_product(y[t:t + 1], w_up[e])
            out[t] += gates[t, j] * fp32_product(silu(up[:, :inner]) * up[:, inner:], w_down[e])[0]
    return out


def random_rows(*shape, scale=1.0, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda") * scale


def distance(got, want):
    return float((got.float() - want).norm() / want.norm())


def run(tokens, hidden, inner, experts, expert_inner, top_k, repeats=0):
    """The dense block (and, up to 64 tokens, the expert block) on random weights:
    {name: (distance from FP32, microseconds or None)}."""
    x = random_rows(tokens, hidden, seed=1).bfloat16()
    stream_rows = random_rows(tokens, hidden, scale=2.0, seed=2).bfloat16()
    weight = 1 + 0.1 * random_rows(hidden, seed=3)
    norm = Norm(weight, tokens)
    y = fp32_norm(x, stream_rows, weight)
    w_up = random_rows(inner, hidden, scale=hidden ** -0.5, seed=4)
    w_down = random_rows(hidden, inner, scale=inner ** -0.5, seed=5)
    blocks = {"dense": (DenseBlock(norm, w_up, w_down), lambda: fp32_dense(y, w_up, w_down))}
    if tokens <= 64 and experts > 0:
        router = random_rows(experts, hidden, scale=hidden ** -0.5, seed=6)
        e_up = random_rows(experts, 2 * expert_inner, hidden, scale=hidden ** -0.5, seed=7)
        e_down = random_rows(experts, hidden, expert_inner, scale=expert_inner ** -0.5, seed=8)
        # the router's choice is made on the rows as the layer gets them
        blocks["experts"] = (ExpertBlock(norm, router, e_up, e_down, top_k),
                             lambda: fp32_experts(norm.y.float(), router, e_up, e_down, top_k))
    result = {}
    for name, (block, reference) in blocks.items():
        out = block(x, stream_rows.clone()).clone()
        status = sg.status()
        if status != sg.OK:
            raise sg.SgemmError(status, name)
        us = None
        if repeats:
            rows = stream_rows.clone()
            start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            for _ in range(3):
                block(x, rows)
            start.record()
            for _ in range(repeats):
                block(x, rows)
            stop.record()
            torch.cuda.synchronize()
            us = start.elapsed_time(stop) * 1e3 / repeats
            block(x, stream_rows.clone())      # the reference reads this block's rows
        result[name] = (distance(out, reference()), us)
    return result


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--expert-inner", type=int, default=1408)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--repeats", type=int, default=50)
    a = ap.parse_args()
    for name, (off, us) in run(a.tokens, a.hidden, a.inner, a.experts, a.expert_inner, a.top_k, a.repeats).items():
        print(f"{name}: {us:.1f} us a block of {a.tokens} tokens, {100 * off:.2f}% from FP32")


if __name__ == "__main__":
    main()
