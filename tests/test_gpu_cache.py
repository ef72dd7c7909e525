"""The attention operators over the 8-bit cache against their 64-bit definitions
(see cache_ref): head norms with rotation, the cache's write and read, and
attention of one new token, over head sizes, group sizes, lengths from none up,
pages that end inside a strip, strides and offsets, masked places that hold NaN,
indices outside their arrays, streams, graphs and several host threads.

Tolerances.  A bf16 result may lie half a unit in the last place (2^-8 relative)
from the definition, besides its FP32 error.  A normalised and rotated element
takes a product with the weight, two products and a difference, relative to
|p_a cos| + |p_b sin| (three roundings of 2^-24 each way), a sum of squares at
most 13 additions deep (half of whose error reaches the root) and four more
roundings: below 16 * 2^-24 = 2^-20.  A scale: the same.  A value read back: one
rounding, 2^-24.  Attention: cache_ref.attend derives its bound.
"""

import threading

import numpy as np
import pytest

import q8_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import cache_ref as ref  # noqa: E402
import dense_fp32_matrix_row_gb300 as sg  # noqa: E402

BF16_HALF = 2.0 ** -8
ROW_TOL = 2.0 ** -20
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


@pytest.fixture(autouse=True)
def clean_status():
    sg.status()
    yield
    torch.cuda.synchronize()
    sg.status()


def close(got, want, tol, dt):
    """Within `tol` plus the output type's rounding; NaN and infinities where the
    definition has them (torch float64 tensors)."""
    got, want, tol = (torch.as_tensor(t, dtype=torch.float64).cpu() for t in (got.double(), want, tol))
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    limit = tol + (BF16_HALF * (1 + 2.0 ** -6) * want.abs() if dt == "bf16" else 0.0) + 2.0 ** -140
    over = torch.where(fine, (got - want).abs() / limit, torch.zeros_like(want))
    assert bool((over <= 1).all()), f"{int((over > 1).sum())} of {over.numel()} off, worst {float(over.max()):.2f}x the bound"


class Rows:
    """(T, H, D) heads as a view of T wider rows: `lead` elements before, `more` behind,
    a pattern in both."""

    def __init__(self, x, dt, lead=0, more=0, offset=0, by_head=False):
        T, H, D = x.shape
        if by_head:
            self.buf = torch.full((offset + H * (T * D + lead) + 8,), 77.0, device="cuda", dtype=DT[dt])
            self.view = torch.as_strided(self.buf, (T, H, D), (D, T * D + lead, 1), offset)
        else:
            ld = lead + H * D + more
            self.buf = torch.full((offset + T * ld + 8,), 77.0, device="cuda", dtype=DT[dt])
            self.view = torch.as_strided(self.buf, (T, H, D), (ld, D, 1), offset + lead)
        self.view.copy_(torch.as_tensor(x).to(DT[dt]))
        self.outside = torch.ones(self.buf.numel(), dtype=torch.bool, device="cuda")
        torch.as_strided(self.outside, (T, H, D), self.view.stride(), self.view.storage_offset()).fill_(False)

    def intact(self):
        return bool((self.buf[self.outside] == 77.0).all())


def f32(t):
    return t.float().cpu().numpy()


def head_sample(rng, T, H, D):
    x = rng.standard_normal((T, H, D))
    x[..., :: max(1, D // 5)] *= 4.0
    return x.astype(np.float32)


def tables(rows, R, seed=0):
    angle = np.arange(rows)[:, None] * (100.0 ** (-2.0 * np.arange(R // 2) / max(R, 1))) + 0.01 * seed
    return torch.from_numpy(np.cos(angle).astype(np.float32)).cuda(), torch.from_numpy(np.sin(angle).astype(np.float32)).cuda()


def vec(rng, D):
    return torch.from_numpy((1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda()


def check_rope(T, Hq, Hk, D, R, dt, norm=True, interleaved=False, lead=0, offset=0, positions=True, in_place=False, x=None,
               by_head=False, table_pad=0):
    rng = np.random.default_rng(T * 1009 + Hq * 101 + Hk * 11 + D + R)
    q, k = (head_sample(rng, T, n, D) if x is None else np.broadcast_to(x, (T, n, D)).copy() for n in (Hq, Hk))
    arrays = [Rows(a, dt, lead, lead, offset, by_head) for a in (q, k)]
    blank = [arrays[i] if in_place else Rows(np.zeros(a.shape, np.float32), dt, lead, 2 * lead, offset, by_head)
             for i, a in enumerate((q, k))]
    kept = [f32(a.view) for a in arrays]
    cos = sin = None
    at = np.arange(T)
    if R:
        cos, sin = tables(2 * T + 5, R + 2 * table_pad)
        cos, sin = cos[:, :R // 2], sin[:, :R // 2]
        if positions:
            at = rng.permutation(2 * T + 5)[:T]
    w = [vec(rng, D) if norm else None for _ in range(2)]
    sg.norm_rope(arrays[0].view if Hq else None, arrays[1].view if Hk else None, cos, sin, blank[0].view if Hq else None,
                 blank[1].view if Hk else None, positions=torch.from_numpy(at).cuda() if R and positions else None,
                 q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=interleaved)
    assert sg.status() == sg.OK
    for i, H in enumerate((Hq, Hk)):
        if H == 0:
            continue
        c, s = (None, None) if not R else (f32(cos)[at], f32(sin)[at])
        _, _, y, size = ref.norm_rope(kept[i], None if w[i] is None else f32(w[i]), c, s, interleaved, 1e-5)
        close(blank[i].view, torch.from_numpy(y), torch.from_numpy(np.nan_to_num(size) * ROW_TOL), dt)
        assert blank[i].intact() and arrays[i].intact()
        if not in_place:
            assert np.array_equal(f32(arrays[i].view), kept[i], equal_nan=True)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,R", [(16, 16), (16, 2), (48, 20), (64, 64), (64, 0), (80, 32), (96, 96), (112, 6), (128, 128),
                                 (128, 64), (144, 144), (192, 8), (256, 256), (256, 100)])
def test_rope(D, R, dt):
    for interleaved in (False, True):
        check_rope(5, 3, 2, D, R, dt, norm=True, interleaved=interleaved)
        check_rope(1, 4, 1, D, R, dt, norm=False, interleaved=interleaved)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (2, 0, 3), (7, 5, 0), (33, 7, 1), (3000, 9, 2)])
def test_rope_counts(T, Hq, Hk, dt):
    """Up to four heads of a token to a group from some 20,000 heads on."""
    check_rope(T, Hq, Hk, 128, 128, dt)
    check_rope(T, Hq, Hk, 80, 48, dt, norm=False, positions=False)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("lead,offset", [(1, 0), (0, 1), (4, 4), (8, 0), (3, 2), (2, 2)])
def test_rope_strides(lead, offset, dt):
    check_rope(4, 3, 2, 64, 64, dt, lead=lead, offset=offset)
    check_rope(4, 3, 2, 64, 64, dt, lead=lead, offset=offset, by_head=True)
    check_rope(4, 3, 2, 64, 32, dt, lead=lead, offset=offset, in_place=True, interleaved=True)
    check_rope(4, 3, 2, 64, 32, dt, table_pad=lead)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["zeros", "huge", "tiny", "nan", "inf", "lowest"])
def test_rope_extremes(kind, dt):
    x = np.ones(64, np.float32)
    x[::3] = -2.0
    x *= {"zeros": 0.0, "huge": 1e25, "tiny": 1e-25}.get(kind, 1.0)
    if kind == "nan":
        x[5] = np.nan
    if kind == "inf":
        x[7] = np.inf
    if kind == "lowest":
        x[:] = -1e38
    check_rope(3, 2, 2, 64, 0, dt, x=x)
    check_rope(3, 2, 2, 64, 64 if kind != "inf" else 0, dt, x=x)


def test_rope_joint_rows_in_place():
    """Queries and keys of a joint projection's rows, each normed in its own place."""
    rng = np.random.default_rng(3)
    T, Hq, Hk, D = 9, 4, 2, 64
    rows = torch.from_numpy(head_sample(rng, T, Hq + 2 * Hk, D)).cuda()
    want = rows.clone()
    cos, sin = tables(T, D)
    w = vec(rng, D)
    a, b = torch.empty((T, Hq, D), device="cuda"), torch.empty((T, Hk, D), device="cuda")
    sg.norm_rope(want[:, :Hq], want[:, Hq:Hq + Hk], cos, sin, a, b, q_weight=w, k_weight=w)
    q, k = rows[:, :Hq], rows[:, Hq:Hq + Hk]
    sg.norm_rope(q, k, cos, sin, q, k, q_weight=w, k_weight=w)
    assert sg.status() == sg.OK
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(rows[:, Hq + Hk:], want[:, Hq + Hk:])


def test_rope_broadcast_input():
    x = torch.randn((1, 1, 64), device="cuda")
    out = torch.empty((6, 3, 64), device="cuda")
    sg.norm_rope(x.expand(6, 3, 64), None, None, None, out, None, q_weight=torch.ones(64, device="cuda"))
    assert sg.status() == sg.OK and torch.equal(out, out[:1, :1].expand(6, 3, 64))


def test_rope_positions_outside_the_tables():
    T, D = 6, 64
    x = torch.randn((T, 3, D), device="cuda")
    cos, sin = tables(4, D)
    at = torch.tensor([0, 4, -1, 3, 1 << 40, 2], device="cuda")
    out = torch.full_like(x, 5.0)
    sg.norm_rope(x, None, cos, sin, out, None, positions=at)
    assert sg.status() == sg.ERR_BAD_INDEX and sg.status() == sg.OK
    good = torch.tensor([0, 3, 5], device="cuda")
    want = torch.empty((3, 3, D), device="cuda")
    sg.norm_rope(x[good], None, cos, sin, want, None, positions=at[good])
    assert torch.equal(out[good], want) and bool((out[[1, 2, 4]] == 5.0).all())


# ---- the cache's write and read ---------------------------------------------------------

def check_write(T, Hk, D, page, dt, rope=True, Hq=0, R=None, interleaved=False, offset=0, lead=0, x=None, pad=0, skip=(),
                beyond=()):
    rng = np.random.default_rng(T * 997 + Hk * 31 + D + page)
    blocks = -(-T // page) + 4
    pool = ref.Pool(blocks, Hk, page, D, seed=T + D, pad=pad)
    before = [t.clone() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale)]
    slots = rng.permutation(blocks * page)[:T].astype(np.int64)
    for t in skip:
        slots[t] = -1 - t
    for t in beyond:
        slots[t] = blocks * page + t
    k, v = (head_sample(rng, T, Hk, D) if x is None else np.broadcast_to(x, (T, Hk, D)).copy() for _ in range(2))
    k, v = Rows(k, dt, lead, lead, offset), Rows(v, dt, lead, 0, offset)
    q = Rows(head_sample(rng, T, Hq, D), dt, lead, lead, offset) if Hq else None
    qo = Rows(np.zeros((T, Hq, D), np.float32), dt, lead, 0, offset) if Hq else None
    cos = sin = c = s = w = None
    if rope:
        R = D if R is None else R
        cos, sin = tables(T, R)
        c, s, w = f32(cos), f32(sin), vec(rng, D)
        sg.norm_rope_write_q8(q.view if Hq else None, k.view, v.view, cos, sin, qo.view if Hq else None, pool.cache(),
                              torch.from_numpy(slots).cuda(), q_weight=w, k_weight=w, eps=1e-5, interleaved=interleaved)
    else:
        sg.cache_write_q8(k.view, v.view, pool.cache(), torch.from_numpy(slots).cuda())
    assert sg.status() == (sg.ERR_BAD_INDEX if len(beyond) else sg.OK)
    stored = np.array([t for t in range(T) if 0 <= slots[t] < blocks * page], dtype=int)
    block, row = slots[stored] // page, slots[stored] % page
    w32 = None if w is None else f32(w)
    for i, (rows, weight, cc, ss) in enumerate(((k, w32, c, s), (v, None, None, None))):
        p32, r, _, _ = ref.norm_rope(f32(rows.view), weight, cc, ss, interleaved, 1e-5)
        nums, scale = ref.quantize(p32, r)
        got = (pool.k, pool.v)[i]
        want = before[i].clone()
        want[block, :, row] = torch.from_numpy(nums[stored].astype(np.int8)).cuda()
        assert torch.equal(got, want), "whole numbers"
        steps = (pool.k_scale, pool.v_scale)[i]
        want = before[2 + i].double()
        want[block, :, row] = torch.from_numpy(scale[stored]).cuda()
        close(steps, want, want.abs().nan_to_num() * ROW_TOL, "fp32")
        rest = torch.ones((blocks, page), dtype=torch.bool, device="cuda")
        rest[block, row] = False
        assert torch.equal(steps.transpose(1, 2)[rest], before[2 + i].transpose(1, 2)[rest])
        assert rows.intact()
    if Hq:
        _, _, y, size = ref.norm_rope(f32(q.view), w32, c, s, interleaved, 1e-5)
        close(qo.view, torch.from_numpy(y), torch.from_numpy(size * ROW_TOL), dt)
        assert qo.intact()
    return pool, slots


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,page", [(16, 1), (48, 5), (64, 16), (80, 20), (112, 3), (128, 16), (128, 64), (192, 7), (256, 32)])
def test_write(D, page, dt):
    check_write(9, 3, D, page, dt, rope=False)
    check_write(9, 3, D, page, dt, Hq=5)
    check_write(1, 2, D, page, dt, Hq=4, R=D // 2, interleaved=True)
    check_write(4, 2, D, page, dt, R=6)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_write_many(dt):
    """Four heads to a group, units of a group that are not full."""
    check_write(2100, 6, 128, 16, dt, Hq=9)
    check_write(4000, 5, 64, 33, dt, rope=False)
    check_write(700, 10, 256, 16, dt, Hq=11, interleaved=True)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("lead,offset,pad", [(1, 0, 0), (0, 1, 1), (4, 4, 2), (0, 0, 5), (3, 2, 0)])
def test_write_strides(lead, offset, pad, dt):
    check_write(6, 2, 64, 16, dt, Hq=4, lead=lead, offset=offset, pad=pad)
    check_write(6, 2, 96, 10, dt, rope=False, lead=lead, offset=offset, pad=pad)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_write_left_out(dt):
    check_write(12, 2, 64, 16, dt, Hq=4, skip=(0, 5, 11))
    check_write(12, 2, 64, 16, dt, rope=False, skip=(3,), beyond=(1, 7))
    check_write(5, 2, 128, 4, dt, skip=(0, 1, 2, 3, 4))


@pytest.mark.parametrize("kind", ["zeros", "huge", "tiny", "nan", "inf"])
def test_write_extremes(kind):
    x = np.ones(64, np.float32)
    x[::3] = -2.0
    x *= {"zeros": 0.0, "huge": 1e25, "tiny": 1e-33}.get(kind, 1.0)
    if kind == "nan":
        x[5] = np.nan
    if kind == "inf":
        x[7] = np.inf
    check_write(3, 2, 64, 16, "fp32", rope=False, x=x)
    check_write(3, 2, 64, 16, "bf16", x=x, R=0)


def test_write_position_outside_the_tables():
    """Such a token is left out altogether: its values are not written either."""
    pool = ref.Pool(2, 2, 8, 64)
    before = [t.clone() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale)]
    x = torch.randn((3, 2, 64), device="cuda")
    out = torch.full_like(x, 5.0)
    cos, sin = tables(4, 64)
    sg.norm_rope_write_q8(x, x.clone(), x.clone(), cos, sin, out, pool.cache(), torch.tensor([0, 1, 2], device="cuda"),
                          positions=torch.tensor([4, -1, 9], device="cuda"))
    assert sg.status() == sg.ERR_BAD_INDEX
    assert bool((out == 5.0).all())
    for t, b in zip((pool.k, pool.v, pool.k_scale, pool.v_scale), before):
        assert torch.equal(t, b)


def test_write_the_same_slot_twice():
    """Its contents are unspecified; nothing else is touched, and what is there is made
    of the tokens that name it."""
    pool = ref.Pool(2, 1, 8, 64)
    before = [t.clone() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale)]
    x = torch.randn((2, 1, 64), device="cuda")
    sg.cache_write_q8(x, x.clone(), pool.cache(), torch.tensor([3, 3], device="cuda"))
    assert sg.status() == sg.OK
    for t, b in zip((pool.k, pool.v, pool.k_scale, pool.v_scale), before):
        mask = torch.ones_like(t, dtype=torch.bool)
        mask[0, :, 3] = False
        assert torch.equal(t[mask], b[mask])
    steps = [float(F / np.float32(127)) for F in f32(x.abs().amax(-1))[:, 0]]
    assert float(pool.k_scale[0, 0, 3]) in steps


def check_read(N, Hk, D, page, dt, lead=0, offset=0, which="kv", pad=0, bad=()):
    rng = np.random.default_rng(N + D + page)
    blocks = -(-N // page) + 2
    pool = ref.Pool(blocks, Hk, page, D, seed=N, pad=pad)
    slots = rng.integers(0, blocks * page, N)           # some of them more than once
    for t in bad:
        slots[t] = -3 if t % 2 else blocks * page
    outs = [Rows(np.full((N, Hk, D), 9.0, np.float32), dt, lead, lead, offset) for _ in range(2)]
    sg.cache_read_q8(pool.cache(), torch.from_numpy(slots).cuda(), outs[0].view if "k" in which else None,
                     outs[1].view if "v" in which else None)
    assert sg.status() == (sg.ERR_BAD_INDEX if any(t % 2 == 0 for t in bad) else sg.OK)
    fine = np.array([t for t in range(N) if t not in bad], dtype=int)
    block, row = slots[fine] // page, slots[fine] % page
    for name, nums, scale, out in (("k", pool.k, pool.k_scale, outs[0]), ("v", pool.v, pool.v_scale, outs[1])):
        want = torch.full((N, Hk, D), 9.0, device="cuda", dtype=torch.float64)
        if name in which:
            want[fine] = nums[block, :, row].double() * scale[block, :, row].double()[..., None]
        close(out.view, want, want.abs() * 2.0 ** -24, dt)
        assert out.intact()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,page", [(16, 1), (64, 16), (80, 20), (128, 16), (192, 7), (256, 32)])
def test_read(D, page, dt):
    check_read(11, 3, D, page, dt)
    check_read(1, 1, D, page, dt, which="v")
    check_read(500, 4, D, page, dt, which="k", pad=1)
    check_read(7, 2, D, page, dt, lead=1, offset=1)
    check_read(7, 5, D, page, dt, lead=8, bad=(0, 1, 6))


# ---- attention --------------------------------------------------------------------------

def check_attend(lens, Hk, G, D, page, dt, window=0, scale=None, q_scale=2.0, pad=0, lead=0, offset=0, seed=0, pool=None,
                 table=None, q=None, width=None, by_head=False, heads=None):
    torch.manual_seed(seed)
    B = len(lens)
    if pool is None:
        pool = ref.Pool(sum(-(-n // page) for n in lens) + 2, Hk, page, D, seed=seed, pad=pad)
        table, kept = pool.table(lens, width, seed)
        pool.poison(kept)
    q = Rows((q_scale * torch.randn((B, Hk * G, D))).numpy() if q is None else q, dt, lead, lead, offset, by_head)
    out = Rows(np.full((B, Hk * G, D), 9.0, np.float32), dt, lead, 0, offset, by_head)
    lse = torch.full((B, Hk * G), 9.0, device="cuda")
    cache, ln = pool.cache(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    sg.attend_q8(q.view, cache, table, ln, out.view, scale=scale, window=window, lse=lse)
    assert sg.status() == sg.OK
    scale = D ** -0.5 if scale is None else scale
    want, tol, want_lse, lse_tol = ref.attend(q.view, pool, table, lens, scale, window, dt == "bf16")
    if heads is None:
        heads = list(range(Hk * G))
    close(out.view[:, heads], want[:, heads], tol[:, heads], dt)
    close(lse[:, heads], want_lse[:, heads], lse_tol[:, heads], "fp32")
    assert out.intact() and q.intact()
    again = torch.empty_like(out.view)
    sg.attend_q8(q.view, cache, table, ln, again, scale=scale, window=window)
    assert torch.equal(again[:, heads], out.view[:, heads]), "the same call gives other bits"
    return out.view


LENS = [1, 0, 2, 15, 16, 17, 31, 63, 64, 65, 0, 127, 128, 129, 300]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 128, 144, 192, 256])
def test_attend(D, dt):
    check_attend(LENS, 2, 4, D, 16, dt)
    check_attend(LENS, 1, 11, D, 32, dt)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [1, 2, 7, 8, 16, 20, 31, 48, 64, 1000])
def test_attend_pages(page, dt):
    check_attend(LENS, 2, 3, 64, page, dt)
    check_attend([5, 200, 33], 1, 2, 128, page, dt, pad=1)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("Hk,G", [(1, 1), (5, 1), (1, 7), (3, 8), (2, 9), (1, 16), (2, 17), (1, 24), (1, 64)])
def test_attend_groups(Hk, G, dt):
    for D in (64, 128, 256):
        check_attend([40, 0, 111], Hk, G, D, 16, dt)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("G", [18, 25, 32, 33, 47, 100])
def test_attend_many_heads_of_a_key_head(G, dt):
    """Up to 32 at a time, in one block and joined from many."""
    for D in (64, 80, 128, 256):
        check_attend([1, 0, 16, 333], 2, G, D, 16, dt)
    check_attend([33, 5000, 70], 1, G, 64, 20, dt, q_scale=1.0)
    check_attend([20000, 3], 1, G, 128, 16, dt, q_scale=1.0, window=17000)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [80, 96, 144, 160, 176, 192, 208])
def test_attend_head_sizes_between(D, dt):
    """Sizes that their form has more room than: chunks and dims behind the head's."""
    for G in (1, 9, 17):
        check_attend([1, 0, 16, 333], 2, G, D, 16, dt)
        check_attend([50, 18], 1, G, D, 20, dt, pad=1)
    check_attend([9000, 3], 2, 5, D, 32, dt, q_scale=1.0)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 5000])
def test_attend_window(window, dt):
    check_attend(LENS + [700], 2, 4, 64, 16, dt, window=window)
    check_attend(LENS + [700], 1, 2, 128, 12, dt, window=window)


def test_attend_window_reads_only_its_pages():
    """Pages before the window may be given away: their entries are not followed, where
    pages end inside a strip too."""
    for page in (16, 5, 24):
        pool = ref.Pool(40, 1, page, 64)
        lens = [37 * page // 2]
        table, _ = pool.table(lens)
        window = 2 * page + 1
        table[0, :(lens[0] - window) // page] = -1
        check_attend(lens, 1, 2, 64, page, "bf16", window=window, pool=pool, table=table)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("Hk,G,D,lens", [(1, 1, 64, [50000]), (1, 8, 128, [40000]), (2, 12, 128, [3, 9000, 0, 2000]),
                                         (1, 4, 256, [20000, 1]), (8, 4, 128, [1025]), (1, 16, 256, [6000]),
                                         (4, 2, 80, [100, 30000, 100])])
def test_attend_long(Hk, G, D, lens, dt):
    """Sequences that several blocks share, up to all of them (parts joined in two steps)."""
    check_attend(lens, Hk, G, D, 16, dt, q_scale=1.0)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_many(dt):
    """More sequences than a block has threads, and than the GPU has blocks."""
    rng = np.random.default_rng(1)
    check_attend([int(n) for n in rng.integers(0, 40, 700)], 1, 2, 64, 16, dt)
    check_attend([int(n) for n in rng.integers(0, 300, 150)], 8, 1, 128, 16, dt)
    check_attend([0] * 400 + [77] + [0] * 400, 1, 2, 64, 16, dt)


def test_attend_very_many():
    """More sequences than a block looks at in one step, most without tokens, the last
    lengths outside the table."""
    B = 152 * 512 + 1000
    pool = ref.Pool(8, 1, 16, 64)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[::1000] = 20
    lens[-2:] = torch.tensor([33, -1], device="cuda")
    table = torch.arange(2, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = torch.randn((1, 2, 64), device="cuda")
    out, lse = torch.full((B, 2, 64), 9.0, device="cuda"), torch.full((B, 2), 9.0, device="cuda")
    sg.attend_q8(q.expand(B, 2, 64), pool.cache(), table, lens, out, lse=lse)
    assert sg.status() == sg.ERR_BAD_INDEX
    want, tol, want_lse, lse_tol = ref.attend(q.repeat(2, 1, 1), pool, table[:2], [20, 32], 0.125, 0, False)
    full = lens == 20
    close(out[full], want[:1].expand(int(full.sum()), 2, 64), tol[:1].expand(int(full.sum()), 2, 64), "fp32")
    close(out[-2:-1], want[1:], tol[1:], "fp32")
    close(lse[-2:-1], want_lse[1:], lse_tol[1:], "fp32")
    none = (lens == 0) | (lens < 0)
    assert float(out[none].abs().max()) == 0 and bool((lse[none] == -float("inf")).all())


def test_attend_no_tokens():
    check_attend([0, 0, 0], 2, 4, 64, 16, "bf16")
    check_attend([0], 1, 1, 128, 8, "fp32", width=0)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("lead,offset,by_head", [(1, 0, False), (0, 1, False), (8, 8, False), (4, 0, True), (3, 3, True)])
def test_attend_strides(lead, offset, by_head, dt):
    check_attend([100, 17, 0, 1], 2, 3, 64, 16, dt, lead=lead, offset=offset, pad=2, by_head=by_head)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("scale,q_scale", [(1.0, 1.0), (0.0, 2.0), (-0.3, 1.0), (1e-20, 1e10), (1e-3, 3e4), (1e20, 1e-21),
                                           (1e36, 1e-36), (1e-37, 3e36), (-1e15, 1e15)])
def test_attend_scales(scale, q_scale, dt):
    """Sharp, flat and turned distributions; queries far outside FP16's range."""
    check_attend([200, 33], 2, 4, 64, 16, dt, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_queries_of_unequal_size(dt):
    """Each head's queries are scaled by themselves; small elements beside large ones."""
    q = np.random.default_rng(2).standard_normal((2, 12, 64)).astype(np.float32)
    q *= (10.0 ** np.arange(-30, 30, 5))[None, :, None].astype(np.float32)
    q[:, :, ::2] *= np.float32(1e-4)
    pool = ref.Pool(20, 3, 16, 64)
    table, _ = pool.table([150, 40])
    for h in range(12):          # one head's scale at a time
        check_attend([150, 40], 3, 4, 64, 16, dt, pool=pool, table=table, q=q, scale=float(10.0 ** (29 - 5 * h)),
                     heads=[h])


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_rising_scores(dt):
    """Scores that grow along the sequence, so that the running maximum moves all the
    way; and that fall."""
    for sign in (1.0, -1.0):
        pool = ref.Pool(20, 1, 16, 64)
        table, _ = pool.table([320])
        pool.k[:] = 100
        order = torch.empty(20, dtype=torch.long, device="cuda")
        order[table[0].long()] = torch.arange(20, device="cuda")
        t = order[:, None] * 16 + torch.arange(16, device="cuda")
        pool.k_scale[:] = (0.0005 * (t + 1)).float()[:, None]
        check_attend([320], 1, 2, 64, 16, dt, pool=pool, table=table, q=np.full((1, 2, 64), sign, np.float32), scale=0.1)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_values_of_unequal_size(dt):
    """Value scales from 1e-30 to 1e30 over the tokens, the small ones first or last, and
    a token of tiny values that takes all the weight."""
    for flip in (False, True):
        pool = ref.Pool(13, 1, 16, 64)
        table, _ = pool.table([200])
        order = torch.empty(13, dtype=torch.long, device="cuda")
        order[table[0].long()] = torch.arange(13, device="cuda")
        t = (order[:, None] * 16 + torch.arange(16, device="cuda")).double()
        t = 199 - t if flip else t
        pool.v_scale[:] = (10.0 ** (t.clamp(0, 199) * 0.3 - 30)).float()[:, None]
        check_attend([200], 1, 2, 64, 16, dt, pool=pool, table=table, q=np.ones((1, 2, 64), np.float32) * 0.1)
    for size in (1e-35, 1e-37, 1e33):       # one warp's and several warps' sequences
        pool = ref.Pool(15, 1, 16, 64)
        table, _ = pool.table([200, 30])
        pool.v_scale.fill_(size)
        check_attend([200, 30], 1, 2, 64, 16, dt, pool=pool, table=table)
    pool = ref.Pool(13, 1, 16, 64)
    table, _ = pool.table([200])
    sink = int(table[0, 0])
    pool.k[sink, 0, 0] = 127
    pool.k_scale[sink, 0, 0] = 1.0
    pool.v_scale[sink, 0, 0] = 1e-4
    check_attend([200], 1, 2, 64, 16, dt, pool=pool, table=table, q=np.full((1, 2, 64), 0.5, np.float32), scale=0.005)


def test_attend_nan_reaches_its_own_readers_only():
    """A NaN row, in one key head of one sequence; a NaN query."""
    pool = ref.Pool(10, 2, 16, 64)
    table, kept = pool.table([40, 60])
    pool.k_scale[int(table[0, 1]), 1, 3] = float("nan")
    q = torch.randn((2, 8, 64), device="cuda")
    q[1, 2, 5] = float("nan")
    q[1, 7, 5] = float("inf")
    out = torch.zeros_like(q)
    sg.attend_q8(q, pool.cache(), table, torch.tensor([40, 60], dtype=torch.int32, device="cuda"), out)
    assert sg.status() == sg.OK
    bad = torch.isnan(out).all(-1)
    want = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    want[0, 4:] = True
    want[1, 2] = want[1, 7] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(out).any(-1), want)
    pool.v_scale[int(table[1, 0]), 0, 0] = float("nan")
    sg.attend_q8(q, pool.cache(), table, torch.tensor([40, 60], dtype=torch.int32, device="cuda"), out)
    assert bool(torch.isnan(out[1, :4]).all()) and not bool(torch.isnan(out[0, :4]).any())


@pytest.mark.parametrize("page", [16, 6])
def test_attend_indices_outside_their_arrays(page):
    pool = ref.Pool(40, 2, page, 64)
    lens = [100, 50, 70]
    table, kept = pool.table(lens)
    pool.poison(kept)
    table[0, 1], table[2, 0] = 40, -1
    out, lse = torch.zeros((3, 4, 64), device="cuda"), torch.zeros((3, 4), device="cuda")
    q = torch.randn((3, 4, 64), device="cuda")
    sg.attend_q8(q, pool.cache(), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse)
    assert sg.status() == sg.ERR_BAD_INDEX and sg.status() == sg.OK
    want, tol, want_lse, lse_tol = ref.attend(q, pool, table, lens, 0.125, 0, False)
    close(out, want, tol, "fp32")
    close(lse, want_lse, lse_tol, "fp32")
    # every page of a sequence outside: no tokens
    table[1] = 1 << 30
    sg.attend_q8(q, pool.cache(), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse)
    assert sg.status() == sg.ERR_BAD_INDEX
    assert bool((out[1] == 0).all()) and bool((lse[1] == -float("inf")).all())


def test_attend_lengths_outside_the_table():
    pool = ref.Pool(20, 1, 16, 64)
    table, _ = pool.table([64, 64, 64])
    q = torch.randn((3, 2, 64), device="cuda")
    out, want = torch.full_like(q, 9.0), torch.empty_like(q)
    sg.attend_q8(q, pool.cache(), table, torch.tensor([-5, 65, 64], dtype=torch.int32, device="cuda"), out)
    assert sg.status() == sg.ERR_BAD_INDEX
    sg.attend_q8(q, pool.cache(), table, torch.tensor([0, 64, 64], dtype=torch.int32, device="cuda"), want)
    assert sg.status() == sg.OK and torch.equal(out, want)


def test_offsets_past_32_bits():
    """A pool of 5 GB of keys: slots, pages and rows at its far end."""
    heads, page, D = 8, 64, 128
    blocks = 5 * (1 << 30) // (heads * page * D)
    k, v = (torch.empty((blocks, heads, page, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((blocks, heads, page), device="cuda") for _ in range(2))
    cache = sg.CacheQ8(k, v, ks, vs)
    last = blocks - 1
    x, y = (torch.randn((page, heads, D), device="cuda") for _ in range(2))
    slots = torch.arange(last * page, blocks * page, device="cuda")
    sg.cache_write_q8(x, y, cache, slots)
    small = sg.CacheQ8(*(t[:1].zero_() for t in (k, v, ks, vs)))
    sg.cache_write_q8(x, y, small, slots - last * page)
    assert sg.status() == sg.OK
    for t in (k, v, ks, vs):
        assert torch.equal(t[last], t[0])
    a, b = torch.empty_like(x), torch.empty_like(x)
    sg.cache_read_q8(cache, slots, a, None)
    sg.cache_read_q8(small, slots - last * page, b, None)
    assert torch.equal(a, b)
    q = torch.randn((1, 16, D), device="cuda")
    got, want = torch.empty_like(q), torch.empty_like(q)
    n = torch.tensor([page - 3], dtype=torch.int32, device="cuda")
    sg.attend_q8(q, cache, torch.tensor([[last]], dtype=torch.int32, device="cuda"), n, got)
    sg.attend_q8(q, small, torch.tensor([[0]], dtype=torch.int32, device="cuda"), n, want)
    assert sg.status() == sg.OK and torch.equal(got, want)


def test_more_tokens_than_a_launch_takes():
    """2^29 and some tokens without a slot (2^30 groups of heads fill a launch), a few
    with one behind them."""
    T, few = (1 << 29) + 77, 5
    pool = ref.Pool(2, 1, 8, 16)
    x = torch.randn((1, 1, 16), device="cuda").bfloat16()
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[-few:] = torch.arange(few, device="cuda")
    sg.cache_write_q8(x.expand(T, 1, 16), x.expand(T, 1, 16), pool.cache(), slots)
    want = ref.Pool(2, 1, 8, 16)
    sg.cache_write_q8(x.expand(few, 1, 16).contiguous(), x.expand(few, 1, 16), want.cache(), slots[-few:].contiguous())
    assert sg.status() == sg.OK
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(pool, n), getattr(want, n))
    out = torch.zeros((T, 1, 16), dtype=torch.bfloat16, device="cuda")
    sg.cache_read_q8(pool.cache(), slots, out, None)
    less = torch.empty((few, 1, 16), dtype=torch.bfloat16, device="cuda")
    sg.cache_read_q8(pool.cache(), slots[-few:].contiguous(), less, None)
    assert sg.status() == sg.OK
    assert torch.equal(out[-few:], less) and float(out[:-few].abs().max()) == 0


# ---- together, streams, graphs, threads ---------------------------------------------------

class Layer:
    """A decoder layer's attention step: heads normed, rotated and stored, then attention."""

    def __init__(self, B, Hk, G, D, page, most, dt=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.B, self.Hk, self.Hq, self.D = B, Hk, Hk * G, D
        width = -(-most // page)
        self.pool = ref.Pool(B * width, Hk, page, D, seed=seed)
        self.cache = self.pool.cache()
        self.table = torch.randperm(B * width, generator=gen, device="cuda").to(torch.int32).view(B, width)
        self.cos, self.sin = tables(most, D)
        self.w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        self.rows = torch.empty((B, self.Hq + 2 * Hk, D), device="cuda", dtype=dt)
        self.q, self.out = (torch.empty((B, self.Hq, D), device="cuda", dtype=dt) for _ in range(2))
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.page = page

    def step(self, stream=None):
        """The rows' tokens become each sequence's next."""
        Hq, Hk = self.Hq, self.Hk
        at = self.lens.long()
        slots = self.table[torch.arange(self.B, device="cuda"), at // self.page].long() * self.page + at % self.page
        self.lens.add_(1)
        sg.norm_rope_write_q8(self.rows[:, :Hq], self.rows[:, Hq:Hq + Hk], self.rows[:, Hq + Hk:], self.cos, self.sin, self.q,
                              self.cache, slots, positions=at, q_weight=self.w, k_weight=self.w, stream=stream)
        sg.attend_q8(self.q, self.cache, self.table, self.lens, self.out, stream=stream)


def reference_layer(layer, tokens):
    """The same steps in 64 bits with whole numbers from FP32: outputs of each step, and
    bounds for them."""
    Hq, Hk, D = layer.Hq, layer.Hk, layer.D
    shadow = ref.Pool(layer.pool.blocks, Hk, layer.page, D)
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(shadow, n).copy_(getattr(layer.pool, n))
    outs = []
    for t, rows in enumerate(tokens):
        x = f32(rows)
        c, s = (f32(a)[t:t + 1].repeat(layer.B, 0) for a in (layer.cos, layer.sin))
        _, _, y, _ = ref.norm_rope(x[:, :Hq], f32(layer.w), c, s, False, 1e-6)
        p32, r, _, _ = ref.norm_rope(x[:, Hq:Hq + Hk], f32(layer.w), c, s, False, 1e-6)
        block, row = layer.table[:, t // layer.page].long(), t % layer.page
        for nums, steps, (q, scale) in ((shadow.k, shadow.k_scale, ref.quantize(p32, r)),
                                        (shadow.v, shadow.v_scale, ref.quantize(x[:, Hq + Hk:], np.ones((layer.B, Hk))))):
            nums[block, :, row] = torch.from_numpy(q.astype(np.int8)).cuda()
            steps[block, :, row] = torch.from_numpy(scale.astype(np.float32)).cuda()
        # the rounding of q to its type moves a score by 2^-8 of its size, like that of out itself
        want, tol, _, _ = ref.attend(torch.from_numpy(y).cuda(), shadow, layer.table, [t + 1] * layer.B, D ** -0.5, 0, True)
        outs.append((want, tol))
    return outs


def test_steps_of_a_layer():
    """Forty tokens decoded one by one.  The query is rounded to bf16 before attention
    reads it: scores of size s move by 2^-8 s (here below 12: 0.05), the weighted sum
    by twice that at most, relative to the weighted magnitudes (at most 4.5)."""
    layer = Layer(3, 2, 4, 64, 16, 48)
    torch.manual_seed(9)
    tokens = [torch.randn_like(layer.rows) for _ in range(40)]
    want = reference_layer(layer, tokens)
    for t, rows in enumerate(tokens):
        layer.rows.copy_(rows)
        layer.step()
        assert sg.status() == sg.OK
        off = (layer.out.double() - want[t][0]).abs()
        assert float((off - want[t][1]).max()) <= 2 * 0.05 * 4.5
        # and on the whole far closer: independent roundings of many elements
        assert float(off.norm() / want[t][0].norm()) < 2.0 ** -5


def test_graph_of_a_step():
    """A captured step replayed for every further token gives what eager steps give; a
    second graph and other calls on the stream do not disturb it."""
    stream = torch.cuda.Stream()
    eager, replayed = Layer(4, 2, 4, 128, 16, 4096, seed=2), Layer(4, 2, 4, 128, 16, 4096, seed=2)
    torch.manual_seed(4)
    tokens = [torch.randn_like(eager.rows) for _ in range(5)]
    start = torch.tensor([0, 700, 3000, 15], dtype=torch.int32, device="cuda")
    graphs = []
    with torch.cuda.stream(stream):
        replayed.rows.copy_(tokens[0])
        replayed.step(stream)                       # sizes the stream's workspace
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                replayed.step(stream)
            graphs.append(g)
    torch.cuda.synchronize()
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(replayed.pool, n).copy_(getattr(eager.pool, n))
    for layer in (eager, replayed):
        layer.lens.copy_(start)
    torch.cuda.synchronize()
    other = Layer(1, 1, 1, 64, 16, 64, seed=5)
    other.rows.normal_()
    for i, rows in enumerate(tokens):
        eager.rows.copy_(rows)
        eager.step()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            replayed.rows.copy_(rows)
            graphs[i % 2].replay()
            other.step(stream)
        assert sg.status(stream) == sg.OK
        assert torch.equal(replayed.out, eager.out)
    del graphs, g
    torch.cuda.synchronize()
    assert sg.release_workspaces() == sg.OK
    eager.lens.copy_(start)
    eager.step()                                    # allocated again
    assert sg.status() == sg.OK


def test_capture_needs_an_eager_call_first():
    assert sg.release_workspaces() == sg.OK
    layer = Layer(1, 1, 2, 64, 16, 64)
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        layer.rows.zero_()
        with pytest.raises(sg.SgemmError) as e:
            sg.attend_q8(layer.q, layer.cache, layer.table, lens, layer.out, stream=stream)
    assert e.value.code == sg.ERR_CAPTURE
    sg.attend_q8(layer.q, layer.cache, layer.table, lens, layer.out, stream=stream)
    assert sg.status(stream) == sg.OK


def test_calls_of_several_threads():
    """Host threads on one stream and on streams of their own: each gets its result."""
    shared = torch.cuda.Stream()
    layers = [Layer(2, 2, 4, 64 * (1 + i % 2), 16, 6000, seed=i) for i in range(4)]
    want, faults = [], []
    for layer in layers:
        layer.q.normal_()
        layer.lens.fill_(5990)
        sg.attend_q8(layer.q, layer.cache, layer.table, layer.lens, layer.out)
        want.append(layer.out.clone())
        layer.out.zero_()
    torch.cuda.synchronize()
    streams = [shared, shared, torch.cuda.Stream(), torch.cuda.Stream()]

    def work(i):
        try:
            layer = layers[i]
            for _ in range(30):
                sg.attend_q8(layer.q, layer.cache, layer.table, layer.lens, layer.out, stream=streams[i])
            streams[i].synchronize()
            if not torch.equal(layer.out, want[i]):
                faults.append(i)
        except Exception as e:      # noqa: BLE001
            faults.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults and sg.status() == sg.OK


# ---- refusals of the binding ------------------------------------------------------------

def test_python_refusals():
    x = torch.zeros((3, 2, 64), device="cuda")
    pool = ref.Pool(4, 2, 16, 64)
    cache, slots = pool.cache(), torch.zeros(3, dtype=torch.int64, device="cuda")
    lens, table = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    cos, sin = tables(8, 64)
    y = torch.zeros_like(x)
    for call in (lambda: sg.norm_rope(x, None, cos, sin, y.bfloat16(), None), lambda: sg.norm_rope(x.half(), None, cos, sin, y, None),
                 lambda: sg.norm_rope(x.cpu(), None, cos, sin, y, None), lambda: sg.norm_rope(x, None, cos, None, y, None),
                 lambda: sg.norm_rope(x, None, cos.double(), sin, y, None),
                 lambda: sg.norm_rope(x, None, cos, sin, y, None, positions=slots.int()),
                 lambda: sg.cache_write_q8(x, x, cache, slots.int()), lambda: sg.cache_write_q8(x, x, cache, None),
                 lambda: sg.cache_write_q8(x, x, pool, slots), lambda: sg.cache_read_q8(cache, slots, y.double()),
                 lambda: sg.attend_q8(x, cache, table.long(), lens, y), lambda: sg.attend_q8(x, cache, table, lens.long(), y),
                 lambda: sg.attend_q8(x, cache, table, lens, y, lse=torch.zeros((3, 2), device="cuda").double()),
                 lambda: sg.CacheQ8(pool.k.float(), pool.v, pool.k_scale, pool.v_scale),
                 lambda: sg.CacheQ8(pool.k, pool.v.cpu(), pool.k_scale, pool.v_scale)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: sg.norm_rope(None, None, cos, sin, None, None), lambda: sg.norm_rope(x, x[:2], cos, sin, y, y[:2]),
                 lambda: sg.norm_rope(x[0], None, cos, sin, y, None), lambda: sg.norm_rope(x, None, cos, sin[:, :3], y, None),
                 lambda: sg.norm_rope(x.transpose(1, 2), None, cos, sin, y.transpose(1, 2), None),
                 lambda: sg.norm_rope(x, None, cos, sin, y, None, q_weight=torch.ones(63, device="cuda")),
                 lambda: sg.cache_write_q8(x[:, :1], x[:, :1], cache, slots), lambda: sg.cache_write_q8(x, x, cache, slots[:2]),
                 lambda: sg.cache_read_q8(cache, slots), lambda: sg.attend_q8(x[:, :1], cache, table, lens, y[:, :1]),
                 lambda: sg.attend_q8(x, cache, table[:2], lens, y), lambda: sg.attend_q8(x, cache, table, lens[:2], y),
                 lambda: sg.CacheQ8(pool.k, pool.v[:2], pool.k_scale, pool.v_scale),
                 lambda: sg.CacheQ8(pool.k.transpose(1, 2), pool.v.transpose(1, 2), pool.k_scale, pool.v_scale)):
        with pytest.raises(ValueError):
            call()
    for call, code in ((lambda: sg.norm_rope(x, None, cos, sin, x[:, :1].expand(3, 2, 64), None), sg.ERR_BAD_LD),
                       (lambda: sg.norm_rope(x, None, cos, sin, y, None, eps=-1.0), sg.ERR_BAD_ARG),
                       (lambda: sg.attend_q8(x, cache, table, lens, x), sg.ERR_ALIAS),
                       (lambda: sg.attend_q8(x, cache, table, lens, y, window=-1), sg.ERR_BAD_ARG),
                       (lambda: sg.attend_q8(x, cache, table, lens, y, scale=float("nan")), sg.ERR_BAD_ARG)):
        with pytest.raises(sg.SgemmError) as e:
            call()
        assert e.value.code == code
    torch.cuda.synchronize()
    assert bool((y == 0).all())


@pytest.mark.parametrize("heads,page,dim", [(0, 16, 64), (2, 0, 64), (2, 16, 0)])
def test_a_cache_without_elements(heads, page, dim):
    k, v = (torch.zeros((4, heads, page, dim), dtype=torch.int8, device="cuda") for _ in range(2))
    with pytest.raises(ValueError):
        sg.CacheQ8(k, v, *(torch.zeros((4, heads, page), device="cuda") for _ in range(2)))


def test_empty_calls():
    pool = ref.Pool(4, 2, 16, 64)
    none = torch.zeros((0, 2, 64), device="cuda")
    slots = torch.zeros(0, dtype=torch.int64, device="cuda")
    cos, sin = tables(8, 64)
    sg.norm_rope(none, none, cos, sin, none.clone(), none.clone(), positions=slots)
    sg.cache_write_q8(none, none, pool.cache(), slots)
    sg.cache_read_q8(pool.cache(), slots, none, none.clone())
    sg.attend_q8(none, pool.cache(), torch.zeros((0, 3), dtype=torch.int32, device="cuda"), slots.int(), none.clone())
    assert sg.status() == sg.OK


def test_a_cache_follows_its_tensors():
    """A tensor that is given another storage is read from there."""
    pool = ref.Pool(4, 2, 16, 64)
    cache = pool.cache()
    slots = torch.arange(5, device="cuda")
    out, want = (torch.empty((5, 2, 64), device="cuda") for _ in range(2))
    other = ref.Pool(6, 2, 16, 64, seed=7)
    sg.cache_read_q8(other.cache(), slots, want)
    pool.k.data, pool.k_scale.data = other.k, other.k_scale
    pool.v.data, pool.v_scale.data = other.v, other.v_scale
    sg.cache_read_q8(cache, slots, out)
    assert torch.equal(out, want)
