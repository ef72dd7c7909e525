"""The attention half of a decoder layer served in 8 bits, weights and cache alike.

What a decoder layer runs in front of its feed-forward block (q8_feed_forward.py),
with every product in 8-bit whole numbers, the residual stream in bfloat16 and the
past keys and values in an 8-bit paged cache:

    h, q     = residual addition, RMS norm and quantisation     (rmsnorm_q8)
    rows     = q @ W_qkv^T: queries, keys and values            (linear_q8)
    Q, cache = head norms and rotation; keys and values stored  (norm_rope_write_q8)
    a        = attention of the new tokens over the cache       (attend_q8)
    out      = a in 8 bits @ W_o^T                              (quantize_q8, linear_q8)

A sequence's first tokens (its prompt) go through the same step, each token a row
with a length of its own; a decode step has one row per sequence.

    python examples/q8_attention.py                       # a decode batch
    python examples/q8_attention.py --sequences 1 --context 32000

prints the time of a step and its distance from the same step in FP32 with
unquantised weights, keys and values.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))]
import dense_fp32_matrix_row_gb300 as sg  # noqa: E402
from q8_feed_forward import Norm, distance, fp32_norm, fp32_product, quantized, random_rows  # noqa: E402


def angles(rows, dim, base=10000.0):
    """(cos, sin) of every position's angles, one column a pair."""
    at = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None]
    turn = at * base ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    return turn.cos().float(), turn.sin().float()


class PagedCache:
    """An 8-bit pool of pages and the sequences' tables into it."""

    def __init__(self, sequences, tokens, kv_heads, dim, page=16):
        width = -(-tokens // page)
        blocks = sequences * width
        self.page = page
        self.cache = sg.CacheQ8(*(torch.zeros((blocks, kv_heads, page, dim), dtype=torch.int8, device="cuda") for _ in range(2)),
                                *(torch.zeros((blocks, kv_heads, page), device="cuda") for _ in range(2)))
        # any order of pages will do
        self.table = torch.randperm(blocks, device="cuda").to(torch.int32).view(sequences, width)

    def slots(self, sequence, position):
        """Where the tokens at these positions of these sequences belong."""
        return self.table[sequence, position // self.page].long() * self.page + position % self.page


class AttentionBlock:
    def __init__(self, norm, w_qkv, w_o, q_weight, k_weight, heads, kv_heads, dim, positions):
        self.norm, self.heads, self.kv_heads, self.dim = norm, heads, kv_heads, dim
        (self.w_qkv, self.s_qkv), (self.w_o, self.s_o) = quantized(w_qkv), quantized(w_o)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.cos, self.sin = angles(positions, dim)
        rows, dev = norm.q.shape[0], w_o.device
        self.joint = torch.empty((rows, heads + 2 * kv_heads, dim), dtype=torch.bfloat16, device=dev)
        self.q, self.a = (torch.empty((rows, heads, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.aq = torch.empty((rows, heads * dim), dtype=torch.int8, device=dev)
        self.a_scale = torch.empty(rows, device=dev)
        self.out = torch.empty((rows, w_o.shape[0]), dtype=torch.bfloat16, device=dev)

    def __call__(self, x, stream_rows, pages, table, slots, positions, lens):
        """One step for as many rows as the block was made for; stream_rows += x in place."""
        n, h, k = self.norm, self.heads, self.kv_heads
        n(x, stream_rows)
        sg.linear_q8(n.q, n.scale, self.w_qkv, self.s_qkv, self.joint.flatten(1))
        sg.norm_rope_write_q8(self.joint[:, :h], self.joint[:, h:h + k], self.joint[:, h + k:], self.cos, self.sin, self.q,
                              pages.cache, slots, positions=positions, q_weight=self.q_weight, k_weight=self.k_weight)
        sg.attend_q8(self.q, pages.cache, table, lens, self.a)
        sg.quantize_q8(self.a.flatten(1), self.aq, self.a_scale)
        sg.linear_q8(self.aq, self.a_scale, self.w_o, self.s_o, self.out)
        return self.out


# ---- the same in FP32 -----------------------------------------------------------------

def fp32_heads(x, weight, cos, sin, eps=1e-6):
    x = x * weight / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    a, b = x.chunk(2, -1)
    c, s = cos[:, None], sin[:, None]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def fp32_rows(y, w_qkv, block, positions):
    """(queries, keys, values) of normalised rows y at these positions."""
    h, k, d = block.heads, block.kv_heads, block.dim
    rows = fp32_product(y, w_qkv).view(-1, h + 2 * k, d)
    cos, sin = block.cos[positions], block.sin[positions]
    return (fp32_heads(rows[:, :h], block.q_weight, cos, sin), fp32_heads(rows[:, h:h + k], block.k_weight, cos, sin),
            rows[:, h + k:])


def fp32_attention(q, k, v):
    """Of one row's queries (heads, dim) over keys and values (tokens, kv_heads, dim)."""
    group = q.shape[0] // k.shape[1]
    q = q.view(k.shape[1], group, -1)
    s = torch.matmul(q, k.permute(1, 2, 0)) / q.shape[-1] ** 0.5
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (torch.matmul(p / p.sum(-1, keepdim=True), v.transpose(0, 1))).flatten()


def run(sequences, context, hidden, heads, kv_heads, dim, repeats=0):
    """A prompt of `context` tokens in each sequence, then a decode step: {name: (distance
    from FP32, microseconds or None)} of the prompt's last tokens and of the step."""
    width = (heads + 2 * kv_heads) * dim
    weight = 1 + 0.1 * random_rows(hidden, seed=1)
    w_qkv = random_rows(width, hidden, scale=hidden ** -0.5, seed=2)
    w_o = random_rows(hidden, heads * dim, scale=(heads * dim) ** -0.5, seed=3)
    q_weight, k_weight = (1.5 + 0.1 * random_rows(dim, seed=s) for s in (4, 5))

    def block(rows):
        return AttentionBlock(Norm(weight, rows), w_qkv, w_o, q_weight, k_weight, heads, kv_heads, dim, context + 1)

    pages = PagedCache(sequences, context + 1, kv_heads, dim)
    tokens = random_rows(sequences, context + 1, hidden, scale=2.0, seed=6).bfloat16()
    zero = torch.zeros((1, hidden), dtype=torch.bfloat16, device="cuda")
    prompt, step = block(context), block(sequences)
    at = torch.arange(context, device="cuda")
    result, keys, values, last = {}, [], [], []
    for b in range(sequences):
        out = prompt(zero.expand(context, hidden).contiguous(), tokens[b, :context].clone(), pages,
                     pages.table[b:b + 1].expand(context, -1).contiguous(), pages.slots(torch.full_like(at, b), at), at,
                     (at + 1).to(torch.int32))
        last.append(out[-1].float())
        y = fp32_norm(zero, tokens[b], weight)
        _, k, v = fp32_rows(y, w_qkv, prompt, torch.arange(context + 1, device="cuda"))
        keys.append(k)
        values.append(v)

    def reference(position):
        y = fp32_norm(zero, tokens[:, position], weight)
        q, _, _ = fp32_rows(y, w_qkv, step, torch.full((sequences,), position, device="cuda"))
        a = torch.stack([fp32_attention(q[b], keys[b][:position + 1], values[b][:position + 1]) for b in range(sequences)])
        return fp32_product(a, w_o)

    result["prompt"] = (distance(torch.stack(last), reference(context - 1)), None)
    new = torch.full((sequences,), context, device="cuda")
    call = (torch.zeros((sequences, hidden), dtype=torch.bfloat16, device="cuda"), tokens[:, context].clone(), pages, pages.table,
            pages.slots(torch.arange(sequences, device="cuda"), new), new, (new + 1).to(torch.int32))
    out = step(*call).clone()
    status = sg.status()
    if status != sg.OK:
        raise sg.SgemmError(status, "step")
    us = None
    if repeats:
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            step(*call)                     # sizes this stream's workspace
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step(*call)
            start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            graph.replay()
            start.record()
            for _ in range(repeats):
                graph.replay()
            stop.record()
        torch.cuda.synchronize()
        us = start.elapsed_time(stop) * 1e3 / repeats
    result["decode"] = (distance(out, reference(context)), us)
    return result


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=16)
    ap.add_argument("--context", type=int, default=2000)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--repeats", type=int, default=50)
    a = ap.parse_args()
    for name, (off, us) in run(a.sequences, a.context, a.hidden, a.heads, a.kv_heads, a.dim, a.repeats).items():
        time = "" if us is None else f"{us:.1f} us a step of {a.sequences} sequences, "
        print(f"{name}: {time}{100 * off:.2f}% from FP32")


if __name__ == "__main__":
    main()
