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
