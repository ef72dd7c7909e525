"""Sizes and strides that the attention operators' argument checks have to let through,
without a GPU: each call here is refused by a later check (an output in an input's
place), so none reaches the CUDA runtime."""

import dense_fp32_matrix_row_gb300 as sg
import pytest
from test_cache_abi import A, attend, fused, heads, pool, read, rope, rotary, write  # noqa: F401
from test_cache_abi import fn  # noqa: F401  (a fixture)


@pytest.mark.parametrize("n,tokens,dim", [(8, 131072, 128), (8, 131088, 128), (8, 262144, 128), (2, 1 << 22, 256),
                                          (32, 1 << 20, 128), (64, 1, 128)])
def test_heads_stored_head_by_head(fn, n, tokens, dim):
    """A head's tokens one behind another: the next head is tokens * dim elements on (or
    more, where the tokens are a part of a long array)."""
    hs = max(tokens, 1 << 20) * dim
    by_head = dict(ld=dim, hs=hs, dim=dim)
    there, more = heads(A[2], n, **by_head), heads(A[2] + 4 * dim, n, **by_head)
    c = pool(heads=n, dim=dim)
    assert read(fn, N=tokens, c=c, k=there, v=None, slots=A[2]) == sg.ERR_ALIAS
    assert rope(fn, T=tokens, D=dim, q=there, qo=more, qw=None, k=None, ko=None, kw=None, rot=None) == sg.ERR_ALIAS
    assert write(fn, T=tokens, k=there, v=there, slots=A[10], c=c) == sg.ERR_ALIAS
    assert attend(fn, B=tokens, q=there, out=more, c=c, pages=1, ldt=1) == sg.ERR_ALIAS


def test_strides_beyond_any_array(fn):
    """heads * hs up to 2^40 elements, whatever the number of heads."""
    for n in (2, 8, 65535):
        most = (1 << 40) // n
        assert rope(fn, T=1, q=heads(A[0], n, hs=most), qo=heads(A[0] + 4 * 64, n, hs=most), k=None, ko=None) == sg.ERR_ALIAS
        assert rope(fn, T=1, q=heads(A[0], n, hs=most + 1), qo=heads(A[1], n), k=None, ko=None) == sg.ERR_BAD_DIM
        assert rope(fn, T=1, q=heads(A[0], n), qo=heads(A[1], n, hs=most + 1), k=None, ko=None) == sg.ERR_BAD_DIM


def test_the_head_stride_of_a_single_head(fn):
    """It leads nowhere: any value will do, in place too."""
    one = pool(heads=1)
    for hs in (0, 7, 1 << 30, (1 << 63) - 1):
        q = heads(A[2], 1, ld=64, hs=hs)
        assert read(fn, c=one, k=q, v=None, slots=A[2]) == sg.ERR_ALIAS
        assert attend(fn, q=q, out=q, c=one) == sg.ERR_ALIAS
        # in its own place, which is allowed: what ends the call is the table in the result's place
        assert rope(fn, q=q, qo=heads(A[2], 1, ld=64, hs=64), qw=None, k=None, ko=None, rot=rotary(cos=A[2])) == sg.ERR_ALIAS


@pytest.mark.parametrize("B,n,key_heads,pages", [(32768, 32, 8, 2048), (256, 128, 8, 65536), (4096, 64, 8, 1000), (33000, 64, 4, 2063),
                                                 (32767, 8, 8, 512), (1, 65535, 1, 8191)])
def test_strips_that_fit_the_list(fn, B, n, key_heads, pages):
    """The list holds a strip of 16 tokens once for a key head's group of 8 query heads or
    more, not once for each query head: rows of a prompt of 32768 tokens and 256
    sequences with tables for a million tokens."""
    q = heads(A[0], n)
    strips = pages + 2
    g = min(n // key_heads, 2 * -(-n // key_heads // 8))
    assert B * key_heads * -(-n // key_heads // 8) * strips < B * key_heads * g * strips < 1 << 31 or n == key_heads
    assert attend(fn, B=B, q=q, out=q, c=pool(heads=key_heads), pages=pages, ldt=pages) == sg.ERR_ALIAS


@pytest.mark.parametrize("B,n,key_heads,pages", [(65536, 32, 8, 4096), (65536, 8, 8, 4096), (1 << 27, 64, 1, 0), (131072, 64, 8, 1022)])
def test_strips_that_do_not(fn, B, n, key_heads, pages):
    q = heads(A[0], n, ld=0)
    assert attend(fn, B=B, q=q, out=heads(A[1], n), c=pool(heads=key_heads), pages=pages, ldt=pages) == sg.ERR_TOO_LARGE


def test_scales_that_are_finite_in_base_2_too(fn):
    """Scores are taken in base 2: a scale that is not finite times log2(e) would make them NaN."""
    for scale in (2.359e38, 2.36e38, 3.4e38, -2.36e38, -3.4e38):
        assert attend(fn, q=heads(A[1], 4), scale=scale) == sg.ERR_BAD_ARG
    for scale in (2.358e38, -2.35e38, 0.0, 1e-45):
        assert attend(fn, q=heads(A[1], 4), scale=scale) == sg.ERR_ALIAS
