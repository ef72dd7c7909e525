"""The attention operators over the 8-bit cache at the ends of their ranges: strides,
counts and magnitudes, and what they report."""

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
