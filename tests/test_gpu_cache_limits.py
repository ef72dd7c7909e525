"""The attention operators over the 8-bit cache at the ends of their ranges: strides,
counts and magnitudes, and what they report."""

import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import cache_ref as ref  # noqa: E402
import dense_fp32_matrix_row_gb300 as sg  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


@pytest.fixture(autouse=True)
def clean_status():
    while sg.status() in (sg.ERR_BAD_INDEX, sg.ERR_TIMEOUT):
        pass
    yield
    torch.cuda.synchronize()
    while sg.status() in (sg.ERR_BAD_INDEX, sg.ERR_TIMEOUT):
        pass


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_long_arrays_stored_head_by_head(dt):
    """131300 tokens of heads of 128: 2^24 elements and more from head to head.  The same
    bits as from rows that lie token by token."""
    T, H, D = 131300, 2, 128
    x = torch.randn((H, T, D), device="cuda").to(dt).transpose(0, 1)
    assert x.stride(1) > 1 << 24
    rows = x.contiguous()
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    angle = torch.rand((T, D // 2), device="cuda")
    cos, sin = angle.cos(), angle.sin()
    got, want = torch.zeros_like(x), torch.empty_like(rows)
    assert got.stride() == x.stride()
    sg.norm_rope(x, None, cos, sin, got, None, q_weight=w)
    sg.norm_rope(rows, None, cos, sin, want, None, q_weight=w)
    assert sg.status() == sg.OK and torch.equal(got, want)

    pools = [ref.Pool(-(-T // 16), H, 16, D) for _ in range(2)]
    slots = torch.arange(T, device="cuda")
    for pool, k in zip(pools, (x, rows)):
        sg.norm_rope_write_q8(None, k, k, cos, sin, None, pool.cache(), slots, k_weight=w)
    assert sg.status() == sg.OK
    for n in ("k", "v", "k_scale", "v_scale"):
        # (the pools' last rows, which no token has, hold the same random numbers)
        assert torch.equal(getattr(pools[0], n), getattr(pools[1], n))
    sg.cache_read_q8(pools[0].cache(), slots, got, None)
    sg.cache_read_q8(pools[0].cache(), slots, want, None)
    assert sg.status() == sg.OK and torch.equal(got, want)

    # a few tokens of such an array as queries and results of attention
    B = 3
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(B, 10)
    lens = torch.tensor([150, 1, 77], dtype=torch.int32, device="cuda")
    sg.attend_q8(x[-B:], pools[0].cache(), table, lens, got[:B])
    sg.attend_q8(rows[-B:], pools[0].cache(), table, lens, want[:B])
    assert sg.status() == sg.OK and torch.equal(got[:B], want[:B])
    sg.norm_rope(x[-1:], None, None, None, got[-1:], None, q_weight=w)
    sg.norm_rope(rows[-1:], None, None, None, want[-1:], None, q_weight=w)
    assert sg.status() == sg.OK and torch.equal(got[-1:], want[-1:])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_of_a_long_prompt(dt):
    """33000 tokens of a prompt, a row each, 8 query heads to a key head and a table for
    32768 tokens: 2^31 strips, were they counted for each query head."""
    B, Hk, G, D, page, pages = 33000, 2, 16, 64, 16, 2048
    pool = ref.Pool(40, Hk, page, D)
    own = torch.randperm(40, device="cuda").to(torch.int32)
    table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
    table[:, :40] = own
    lens = (torch.arange(B, device="cuda") % 60 + 1).to(torch.int32)
    lens[-1], lens[1000] = 40 * page, 0
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q = torch.randn((B, Hk * G, D), device="cuda", generator=gen).to(dt)
    out, lse = torch.full_like(q, 9.0), torch.full((B, Hk * G), 9.0, device="cuda")
    assert B * Hk * G * (pages + 2) > 1 << 31
    sg.attend_q8(q, pool.cache(), table, lens, out, lse=lse)
    assert sg.status() == sg.OK
    some = [0, 1, 59, 999, 1000, 1001, 16384, 32767, 32768, B - 2, B - 1]
    want, tol, want_lse, lse_tol = ref.attend(q[some], pool, table[some], lens[some].tolist(), D ** -0.5, 0, dt == torch.bfloat16)
    # (a bf16 result is rounded by half a unit in its last place)
    tol = tol + (2.0 ** -8 * (1 + 2.0 ** -6) * want.abs() if dt == torch.bfloat16 else 0)
    assert bool(((out[some].double() - want).abs() <= tol + 2.0 ** -140).all())
    none = want_lse.isinf()
    assert torch.equal(lse[some].isinf(), none) and bool(((lse[some].double() - want_lse).abs() <= lse_tol)[~none].all())
    assert bool(out.isfinite().all()) and not bool((out == 9.0).all(-1).any())


# ---- tensors of a cache that change ---------------------------------------------------

def four(blocks, heads, page, dim, more=0):
    """Zeroed tensors of a cache; pages `more` rows of all heads further apart."""
    def one(tail, dtype):
        t = torch.zeros((blocks, heads * (page + more)) + tail, dtype=dtype, device="cuda")
        return t[:, :heads * page].view(blocks, heads, page, *tail)
    return [one((dim,), torch.int8), one((dim,), torch.int8), one((), torch.float32), one((), torch.float32)]


def stored(cache, slots, x):
    sg.cache_write_q8(x, x, cache, slots)
    out = torch.zeros_like(x)
    sg.cache_read_q8(cache, slots, None, out)
    assert sg.status() == sg.OK
    return out


def give(tensors, others):
    for t, other in zip(tensors, others):
        t.data = other


@pytest.mark.parametrize("kind", ["pages", "strides", "heads"])
def test_a_cache_follows_its_tensors_layout(kind):
    """Tensors that get another shape or other strides at the same address are used as
    they then are: what a new CacheQ8 around them would give."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    old = four(6, 2, 16, 64, more=8)
    cache = sg.CacheQ8(*old)
    x = torch.randn((30, 2, 64), device="cuda", generator=gen)
    slots = torch.randperm(48, device="cuda", generator=gen)[:30]
    stored(cache, slots, x)
    whole = [t.as_strided((6 * 2 * 24,) + t.shape[3:], (t.stride(2),) + t.stride()[3:]) for t in old]   # all rows there are
    shape, strided = {"pages": ((12, 2, 8), 24), "strides": ((6, 2, 16), 40), "heads": ((6, 1, 16), 48)}[kind]
    new = [w.as_strided(shape + w.shape[1:], tuple(n * w.stride(0) for n in (strided, shape[2], 1)) + w.stride()[1:])
           for w in whole]
    if kind == "heads":
        x = x[:, :1].contiguous()
    for w in whole:
        w.zero_()
    give(old, new)
    assert old[0].data_ptr() == whole[0].data_ptr()
    got = stored(cache, slots, x)
    seen = [w.clone() for w in whole]
    for w in whole:
        w.zero_()
    want = stored(sg.CacheQ8(*new), slots, x)
    assert torch.equal(got, want) and bool(got.any())
    for a, b in zip(seen, whole):
        assert torch.equal(a, b)
    assert (cache.heads, cache.page, cache.slots) == (shape[1], shape[2], shape[0] * shape[2])


def test_a_cache_that_has_shrunk():
    """Slots and pages behind its end are outside it, though their memory is still there."""
    tensors = four(8, 1, 16, 64)
    kept = [t.detach() for t in tensors]
    cache = sg.CacheQ8(*tensors)
    x = torch.randn((2, 1, 64), device="cuda")
    stored(cache, torch.tensor([3, 100], device="cuda"), x)
    give(tensors, [t[:2] for t in kept])
    before = [t.clone() for t in kept]
    sg.cache_write_q8(x + 1, x, cache, torch.tensor([32, 127], device="cuda"))
    assert sg.status() == sg.ERR_BAD_INDEX
    q, out = torch.randn((1, 2, 64), device="cuda"), torch.full((1, 2, 64), 9.0, device="cuda")
    sg.attend_q8(q, cache, torch.tensor([[6]], dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda"), out)
    assert sg.status() == sg.ERR_BAD_INDEX and float(out.abs().max()) == 0
    for a, b in zip(before, kept):
        assert torch.equal(a, b)


def test_a_cache_with_a_tensor_replaced():
    a, b = four(4, 2, 16, 64), four(9, 2, 16, 64)
    cache = sg.CacheQ8(*a)
    x = torch.randn((5, 2, 64), device="cuda")
    slots = torch.arange(60, 65, device="cuda")         # the second pool alone has them all
    cache.k, cache.v = b[0], b[1]
    with pytest.raises(ValueError):                     # scales of another number of pages
        sg.cache_write_q8(x, x, cache, slots)
    with pytest.raises(ValueError):
        sg.cache_write_q8(x, x, cache, slots)
    cache.k_scale, cache.v_scale = b[2], b[3]
    got = stored(cache, slots, x)
    assert cache.slots == 9 * 16
    want = stored(sg.CacheQ8(*four(9, 2, 16, 64)), slots, x)
    assert torch.equal(got, want) and bool((b[0] != 0).any()) and not bool(a[0].any())
    cache.k = cache.v = cache.k_scale = cache.v_scale = None
    with pytest.raises(TypeError):
        sg.cache_write_q8(x, x, cache, slots)


# ---- what is reported -----------------------------------------------------------------

def test_status_tells_both_kinds():
    """A time-out and an index outside its array, whichever came first."""
    x = torch.randn((1, 2, 64), device="cuda")
    tables = torch.ones((4, 32), device="cuda")
    out = torch.empty_like(x)

    def bad_index():
        sg.norm_rope(x, None, tables, tables, out, None, positions=torch.tensor([9], device="cuda"))

    def timeout():
        assert sg.selftest_wait(1000) == sg.OK

    for calls in ((bad_index, timeout), (timeout, bad_index), (timeout, bad_index, bad_index, timeout)):
        for call in calls:
            call()
        assert [sg.status() for _ in range(3)] == [sg.ERR_TIMEOUT, sg.ERR_BAD_INDEX, sg.OK]
    bad_index()
    assert [sg.status() for _ in range(2)] == [sg.ERR_BAD_INDEX, sg.OK]
    timeout()
    other = torch.cuda.Stream()
    assert [sg.status(other) for _ in range(2)] == [sg.ERR_TIMEOUT, sg.OK]


# ---- values of unequal size -----------------------------------------------------------

def products_bound(q, pool, table, lens, scale, bf16):
    """(out, tol, lse, lse_tol) as cache_ref.attend gives them (its bounds are derived there),
    but for the last term of tol: what FP16's smallest step leaves off a product
    p * (value scale) goes by the head's largest such product, not by the largest scale.  In
    the kernel's units the largest is at 2^8 or more and the step 2^-24, so each product is
    off by at most 2^-33 of the largest, times a whole number of up to 127.  Where products
    are below 2^-53 of (largest p) * (largest scale), sums of p end that: p is held up to
    2^60, scales up to 2^8 or more, and the step is 2^-93 of them."""
    _, _, lse, lse_tol = ref.attend(q, pool, table, lens, scale, 0, bf16)
    B, H, D = q.shape
    Hk, u, d = pool.heads, 2.0 ** -23, torch.float64
    out, tol = (torch.zeros((B, H, D), dtype=d, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        block, row = table[b].long()[t // pool.page], t % pool.page
        k = pool.k[block, :, row].to(d) * pool.k_scale[block, :, row].to(d)[..., None]
        steps = pool.v_scale[block, :, row].to(d)                           # (n, Hk)
        v = pool.v[block, :, row].to(d) * steps[..., None]
        x = q[b].to(d).view(Hk, H // Hk, D)
        s = torch.einsum("hgd,nhd->hgn", x, k) * scale
        size = torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()) * abs(scale)
        p = torch.softmax(s, -1)
        out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(H, D)
        eps = (10 + D / 8) * u * size.amax(-1) + 6 * u
        weight = torch.einsum("hgn,nhd->hgd", p, v.abs())
        product = (p * steps.abs().T[:, None]).amax(-1)                     # (Hk, G)
        least = 127 * n * (2.0 ** -33 * product + 2.0 ** -93 * steps.abs().amax(0)[:, None])
        tol[b] = (weight * (2 * eps + 2 * (n / 16 + 24) * u + (2.0 ** -11 if bf16 else 2.0 ** -21))[..., None]
                  + least[..., None]).reshape(H, D)
    return out, tol, lse, lse_tol


def check_products(q, pool, table, lens, scale):
    bf16 = q.dtype == torch.bfloat16
    out, lse = torch.full_like(q, 9.0), torch.zeros(q.shape[:2], device="cuda")
    sg.attend_q8(q, pool.cache(), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, scale=scale, lse=lse)
    assert sg.status() == sg.OK
    want, tol, want_lse, lse_tol = products_bound(q, pool, table, lens, scale, bf16)
    tol = tol + (2.0 ** -8 * (1 + 2.0 ** -6) * want.abs() if bf16 else 0) + 2.0 ** -140
    over = (out.double() - want).abs() / tol
    assert bool((over <= 1).all()), f"{int((over > 1).sum())} of {over.numel()} off, worst {float(over.max()):.3g}x the bound"
    assert bool(((lse.double() - want_lse).abs() <= lse_tol).all())


def scored(pool, table, lens, score, size):
    """Gives token t of sequence b the score score[b][t] for a query of ones (in its first
    dim alone) and scale 1, and the value scale size[b][t], for each key head."""
    pool.k.zero_()
    pool.k[..., 0] = 100
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        block, row = table[b].long()[t // pool.page], t % pool.page
        pool.k_scale[block, :, row] = (score[b].to("cuda") / 100).float()[:, None]
        pool.v_scale[block, :, row] = size[b].to("cuda").float()[:, None]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,G", [(64, 4), (64, 12), (96, 7), (128, 8), (128, 24), (192, 5), (256, 8), (256, 3)])
def test_small_values_of_large_weight(D, G, dt):
    """Value scales over fifty powers of two, the smaller the more weight: heads that turn
    the scores up, down or off."""
    lens = [200, 90, 5000, 16, 7]
    gen = torch.Generator()
    gen.manual_seed(D + G)
    pool = ref.Pool(sum(-(-n // 16) for n in lens) + 1, 2, 16, D, seed=G)
    table, kept = pool.table(lens)
    fall = [50 * torch.rand(n, generator=gen, dtype=torch.float64) for n in lens]
    turn = [0.8 + 0.4 * torch.rand(n, generator=gen, dtype=torch.float64) for n in lens]
    scored(pool, table, lens, [0.6931 * a * w for a, w in zip(fall, turn)], [2.0 ** -a for a in fall])
    pool.poison(kept)
    q = torch.zeros((len(lens), 2 * G, D), device="cuda")
    q[..., 0] = torch.linspace(-0.5, 1.0, 2 * G, device="cuda")
    check_products(q.to(dt), pool, table, lens, 1.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ratio", [2.0 ** -11, 2.0 ** -16, 2.0 ** -24, 2.0 ** -36, 2.0 ** -44, 0.0])
@pytest.mark.parametrize("at", [(0, 3), (3, 0), (2, 40), (40, 2), (17, 150)])
def test_one_small_value_beside_a_large_one(at, ratio, dt):
    """All weight on a token whose values are `ratio` of another's, which comes before it,
    behind it, or in its strip of 16; more tokens like it follow."""
    n = 160         # ten strips: one warp's
    pool = ref.Pool(12, 1, 16, 64, seed=3)
    table, _ = pool.table([n])
    score, size = torch.zeros(n, dtype=torch.float64), torch.full((n,), ratio / 2, dtype=torch.float64)
    small, large = at
    score[small], size[small] = 50.0, ratio
    score[100:103], size[100:103] = 50.0, ratio
    size[large] = 1.0
    scored(pool, table, [n], [score], [size])
    q = torch.zeros((1, 4, 64), device="cuda")
    q[..., 0] = torch.tensor([1.0, 0.9, 0.0, -1.0], device="cuda")
    check_products(q.to(dt), pool, table, [n], 1.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_values_that_grow_while_scores_fall(dt):
    """Each strip's values are larger and its scores lower than the last one's, and the
    other way round: every strip changes how products are scaled."""
    n = 160
    for sign in (1, -1):
        for slope in (0.5, 1.0, 1.5):
            pool = ref.Pool(12, 1, 16, 128, seed=4)
            table, _ = pool.table([n])
            t = torch.arange(n, dtype=torch.float64)
            t = t if sign > 0 else n - 1 - t
            scored(pool, table, [n], [-0.6931 * slope * t], [2.0 ** (t - 100)])
            q = torch.zeros((1, 3, 128), device="cuda")
            q[..., 0] = torch.tensor([1.0, 0.75, 0.25], device="cuda")
            check_products(q.to(dt), pool, table, [n], 1.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,D,lens", [(4, 64, [30, 1]), (9, 96, [200, 17]), (8, 128, [5000, 160]), (20, 128, [40, 9000]),
                                      (8, 192, [3000]), (4, 256, [16000]), (1, 64, [60000])])
def test_values_near_the_end_of_the_range(G, D, lens, dt):
    """Sums of values that pass FP32's range, whose mean does not: one warp's, several
    warps', several blocks'."""
    pool = ref.Pool(sum(-(-n // 16) for n in lens) + 1, 1, 16, D, seed=D)
    table, kept = pool.table(lens)
    pool.v.copy_(pool.v // 16 + 100)            # 92 to 107
    pool.v_scale.copy_(3e36 * (0.9 + 0.1 * torch.rand_like(pool.v_scale)))
    pool.poison(kept)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    q = torch.randn((len(lens), G, D), device="cuda", generator=gen).to(dt)
    check_products(q, pool, table, lens, D ** -0.5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_values_of_all_sizes_in_one_sequence(dt):
    """Runs of 300 tokens from 1e-33 to 3e36, in several blocks: parts that are scaled
    differently are joined, whichever have the weight."""
    lens, D = [9000], 128
    n = lens[0]
    for slope in (0.0, 1.0, -1.0):
        pool = ref.Pool(570, 2, 16, D, seed=8)
        table, _ = pool.table(lens)
        run = (torch.arange(n) // 300).double()         # 0 to 29
        size = 3e36 * 10.0 ** (-69 * run / 29)
        scored(pool, table, lens, [slope * 2.0 * run], [size])
        q = torch.zeros((1, 10, D), device="cuda")
        q[..., 0] = torch.linspace(0.2, 1.0, 10, device="cuda")
        check_products(q.to(dt), pool, table, lens, 1.0)


# ---- host threads ---------------------------------------------------------------------

def test_every_call_of_several_threads():
    """Threads on one stream and on streams of their own, sequences that many blocks share
    (parts and counters in the streams' workspaces): each call's own result, in arrays of
    its own, is compared."""
    calls, lens = 40, [[5990, 3000], [11, 7000], [6000, 1], [2500, 2500]]
    shared = torch.cuda.Stream()
    streams = [shared, shared, torch.cuda.Stream(), torch.cuda.Stream()]
    work, want = [], []
    for i in range(4):
        Hk, G, D = (2, 4, 64) if i % 2 else (1, 12, 128)
        pool = ref.Pool(sum(-(-n // 16) for n in lens[i]), Hk, 16, D, seed=i)
        table, _ = pool.table(lens[i], seed=i)
        q = torch.randn((2, Hk * G, D), device="cuda").bfloat16()
        outs = torch.full((calls,) + q.shape, float("nan"), device="cuda", dtype=q.dtype)
        lses = torch.full((calls,) + q.shape[:2], float("nan"), device="cuda")
        args = (q, pool.cache(), table, torch.tensor(lens[i], dtype=torch.int32, device="cuda"))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        sg.attend_q8(*args, out, lse=lse)
        work.append((args, outs, lses))
        want.append((out, lse))
    torch.cuda.synchronize()
    begin, faults = threading.Barrier(4), []

    def run(i):
        try:
            args, outs, lses = work[i]
            begin.wait(60)
            for k in range(calls):
                sg.attend_q8(*args, outs[k], lse=lses[k], stream=streams[i])
            streams[i].synchronize()
        except Exception as e:      # noqa: BLE001
            faults.append(repr(e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults and sg.status() == sg.OK
    for (_, outs, lses), (out, lse) in zip(work, want):
        assert torch.equal(outs, out.expand_as(outs)) and torch.equal(lses, lse.expand_as(lses))


# ---- batches with gaps ----------------------------------------------------------------

def test_sequences_among_empty_ones():
    """Gaps of all sizes between sequences of one warp and of several."""
    gen = torch.Generator()
    gen.manual_seed(6)
    for gap in (1, 2, 31, 32, 33, 64, 100):
        lens = []
        for n in torch.randint(1, 90, (60,), generator=gen).tolist():
            lens += [n] + [0] * gap
        lens += [1, 0]
        pool = ref.Pool(sum(-(-n // 16) for n in lens) + 1, 1, 16, 64, seed=gap)
        table, kept = pool.table(lens)
        pool.poison(kept)
        q = torch.randn((len(lens), 3, 64), device="cuda").bfloat16()
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
        sg.attend_q8(q, pool.cache(), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse)
        assert sg.status() == sg.OK
        want, tol, want_lse, lse_tol = ref.attend(q, pool, table, lens, 0.125, 0, True)
        assert bool(((out.double() - want).abs() <= tol + 2.0 ** -8 * (1 + 2.0 ** -6) * want.abs() + 2.0 ** -140).all())
        none = want_lse.isinf()
        assert torch.equal(lse.isinf(), none) and bool(((lse.double() - want_lse).abs() <= lse_tol)[~none].all())


def test_time_of_wide_gaps():
    """Short sequences at both ends and in the middle of a million rows: a warp that goes on
    behind a gap looks at 32 rows at a time.  That is 2^14 loads one after the other, 33 ms were
    each of them 2 us long (12 ms in all where measured); one row at a time it was 87 ms."""
    B = 1 << 20
    pool = ref.Pool(2, 1, 16, 64)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for first, n in ((0, 4001), (B // 2, 4003), (B - 3999, 3999)):
        lens[first:first + n] = 9
    table = torch.arange(2, dtype=torch.int32, device="cuda").expand(B, 2).contiguous()
    q = torch.randn((1, 2, 64), device="cuda").bfloat16().expand(B, 2, 64)
    out = torch.full((B, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    sg.attend_q8(q, pool.cache(), table, lens, out)         # sizes the workspace
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    sg.attend_q8(q, pool.cache(), table, lens, out)
    stop.record()
    assert sg.status() == sg.OK
    there = lens > 0
    assert bool(out[0].any()) and torch.equal(out[there], out[:1].expand(int(there.sum()), 2, 64)) and not bool(out[~there].any())
    assert start.elapsed_time(stop) < 50
