"""Argument checks of the attention operators through the C ABI, without a GPU: no
call here is accepted, so none reaches the CUDA runtime (pointers are plain
numbers), except empty ones, which return before it."""

import dense_fp32_matrix_row_gb300 as sg
import pytest

A = [i << 34 for i in range(1, 20)]      # arrays far apart
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fn():
    sg.build()
    from dense_fp32_matrix_row_gb300 import q8
    return lambda name, *a: q8._entry(name)(*a)


def heads(p, n, ld=None, hs=64, dim=64):
    from dense_fp32_matrix_row_gb300 import cache
    return cache._HEADS(p, n, n * dim if ld is None else ld, hs)


def rotary(cos=A[6], sin=A[7], rows=100, ld=32, dims=64, positions=A[8], interleaved=0):
    from dense_fp32_matrix_row_gb300 import cache
    return cache._ROTARY(cos, sin, rows, ld, dims, positions, interleaved)


def pool(k=A[10], v=A[11], ks=A[12], vs=A[13], blocks=9, heads=2, page=16, dim=64, strides=None):
    from dense_fp32_matrix_row_gb300 import cache
    rows = heads * page
    return cache._CACHE(k, v, ks, vs, blocks, heads, page, dim, *(strides or (rows * dim, rows * dim, rows, rows)))


Q, QO, K, KO, V = heads(A[0], 4), heads(A[1], 4), heads(A[2], 2), heads(A[3], 2), heads(A[4], 2)


def rope(fn, T=3, D=64, type_=0, q=Q, qo=QO, qw=A[14], k=K, ko=KO, kw=A[15], eps=1e-6, rot="default"):
    return fn("sgemm_norm_rope", T, D, type_, q, qo, qw, k, ko, kw, eps, rotary() if rot == "default" else rot, None)


def write(fn, T=3, type_=0, k=K, v=V, slots=A[9], c="default"):
    return fn("sgemm_q8_cache_write", T, type_, k, v, slots, pool() if c == "default" else c, None)


def fused(fn, T=3, type_=0, q=Q, qo=QO, qw=A[14], k=K, kw=A[15], v=V, eps=1e-6, rot="default", slots=A[9], c="default"):
    return fn("sgemm_q8_norm_rope_write", T, type_, q, qo, qw, k, kw, v, eps, rotary() if rot == "default" else rot,
              slots, pool() if c == "default" else c, None)


def read(fn, N=3, type_=0, c="default", slots=A[9], k=K, v=V):
    return fn("sgemm_q8_cache_read", N, type_, pool() if c == "default" else c, slots, k, v, None)


def attend(fn, B=3, type_=0, q=Q, c="default", table=A[5], ldt=8, pages=8, lens=A[6], scale=0.1, window=0, out=QO,
           lse=A[7]):
    return fn("sgemm_q8_attend", B, type_, q, pool() if c == "default" else c, table, ldt, pages, lens, scale, window,
              out, lse, None)


def test_rope_refusals(fn):
    assert rope(fn, T=-1) == rope(fn, T=1 << 31) == sg.ERR_BAD_DIM
    for d in (0, 8, 24, 272, -16):
        assert rope(fn, D=d) == sg.ERR_BAD_DIM
    assert rope(fn, type_=2) == rope(fn, eps=-1.0) == rope(fn, eps=NAN) == sg.ERR_BAD_ARG
    assert rope(fn, qo=None) == rope(fn, ko=None) == rope(fn, q=heads(0, 4)) == sg.ERR_NULL_PTR
    assert rope(fn, qo=heads(A[1], 5)) == rope(fn, ko=heads(A[3], 1)) == rope(fn, q=heads(A[0], -1)) == sg.ERR_BAD_DIM
    assert rope(fn, q=heads(A[0], 65536), qo=heads(A[1], 65536)) == sg.ERR_BAD_DIM
    # strides: negative; an output whose elements share a place
    assert rope(fn, q=heads(A[0], 4, ld=-1)) == rope(fn, q=heads(A[0], 4, hs=-64)) == sg.ERR_BAD_LD
    assert rope(fn, qo=heads(A[1], 4, ld=255)) == rope(fn, qo=heads(A[1], 4, hs=63)) == sg.ERR_BAD_LD
    assert rope(fn, qo=heads(A[1], 4, ld=64, hs=3 * 64 - 1)) == sg.ERR_BAD_LD
    assert rope(fn, q=heads(A[0], 4, ld=1 << 50)) == sg.ERR_BAD_DIM
    assert rope(fn, q=heads(A[0] + 2, 4)) == rope(fn, qw=A[14] + 1) == rope(fn, qo=heads(A[1] + 1, 4), type_=1) == sg.ERR_BAD_ARG
    assert rope(fn, T=0, q=None) == sg.OK and rope(fn, q=None, k=None) == sg.OK


def test_rope_table_refusals(fn):
    assert rope(fn, rot=rotary(dims=65)) == rope(fn, rot=rotary(dims=66)) == rope(fn, rot=rotary(dims=-2)) == sg.ERR_BAD_DIM
    assert rope(fn, rot=rotary(rows=-1)) == rope(fn, rot=rotary(rows=2, positions=0)) == sg.ERR_BAD_DIM
    assert rope(fn, rot=rotary(cos=0)) == rope(fn, rot=rotary(sin=0)) == sg.ERR_NULL_PTR
    assert rope(fn, rot=rotary(ld=31)) == sg.ERR_BAD_LD
    assert rope(fn, rot=rotary(cos=A[6] + 2)) == rope(fn, rot=rotary(positions=A[8] + 4)) == sg.ERR_BAD_ARG


def test_rope_aliases(fn):
    for name in (A[0] + 64 * 4, A[2], A[6], A[7], A[8], A[14], A[15], A[3]):
        assert rope(fn, qo=heads(name, 4)) == sg.ERR_ALIAS, hex(name)
    # in place only with the same strides, and each result in its own input's place
    assert rope(fn, qo=heads(A[0], 4, ld=512)) == sg.ERR_ALIAS
    assert rope(fn, q=heads(A[0], 2), qo=heads(A[1], 2), k=heads(A[2], 2), ko=heads(A[0], 2)) == sg.ERR_ALIAS
    # rows of a joint projection: heads apart from one another, and heads that meet
    joint = dict(q=heads(A[0], 4, ld=512), k=heads(A[0] + 4 * 256, 2, ld=512))
    assert rope(fn, **joint, qo=heads(A[0] + 4 * 128, 4, ld=512), ko=KO) == sg.ERR_ALIAS
    assert rope(fn, **joint, qo=QO, ko=heads(A[0] + 4 * 448, 2, ld=512)) == sg.ERR_ALIAS


def test_write_refusals(fn):
    for call in (write, fused):
        assert call(fn, T=-1) == sg.ERR_BAD_DIM
        assert call(fn, type_=3) == sg.ERR_BAD_ARG
        assert call(fn, k=None) == call(fn, v=None) == call(fn, slots=None) == call(fn, c=None) == sg.ERR_NULL_PTR
        assert call(fn, k=heads(A[2], 3)) == call(fn, v=heads(A[4], 1)) == sg.ERR_BAD_DIM
        assert call(fn, slots=A[9] + 4) == sg.ERR_BAD_ARG
        assert call(fn, k=heads(A[2] + 1, 2)) == sg.ERR_BAD_ARG
        for place in (A[10], A[11] + 9 * 2048 - 1, A[12], A[13] + 4 * 9 * 32 - 4):
            aligned = place // 4 * 4
            assert call(fn, k=heads(aligned, 2)) == call(fn, v=heads(aligned, 2)) == sg.ERR_ALIAS
        assert call(fn, slots=A[12]) == sg.ERR_ALIAS
        assert call(fn, T=0, k=None, v=None, slots=None) == sg.OK
    assert fused(fn, qo=None) == sg.ERR_NULL_PTR and fused(fn, eps=-1.0) == sg.ERR_BAD_ARG
    assert fused(fn, qo=heads(A[10], 4)) == fused(fn, qo=heads(A[4], 4)) == fused(fn, kw=A[13]) == sg.ERR_ALIAS
    assert fused(fn, rot=rotary(cos=A[11])) == sg.ERR_ALIAS


@pytest.mark.parametrize("call", [write, fused, read, attend])
def test_cache_refusals(fn, call):
    for bad in (dict(dim=24), dict(dim=0), dict(dim=272), dict(blocks=-1), dict(heads=0), dict(page=0),
                dict(page=(1 << 30) + 1), dict(blocks=1 << 41), dict(heads=65536)):
        assert call(fn, c=pool(**bad)) == sg.ERR_BAD_DIM, bad
    assert call(fn, c=pool(heads=2, page=1 << 30)) == sg.ERR_BAD_DIM
    for bad in (dict(k=0), dict(v=0), dict(ks=0), dict(vs=0)):
        assert call(fn, c=pool(**bad)) == sg.ERR_NULL_PTR, bad
    for i, least in enumerate((2048, 2048, 32, 32)):
        strides = [2048, 2048, 32, 32]
        strides[i] = least - 1
        assert call(fn, c=pool(strides=strides)) == sg.ERR_BAD_LD
        strides[i] = 1 << 45
        assert call(fn, c=pool(strides=strides)) == sg.ERR_BAD_DIM
    assert call(fn, c=pool(strides=(2056, 2048, 32, 32))) == call(fn, c=pool(k=A[10] + 8)) == sg.ERR_BAD_ARG
    assert call(fn, c=pool(vs=A[13] + 2)) == sg.ERR_BAD_ARG


def test_cache_arrays_overlap(fn):
    assert write(fn, c=pool(v=A[10] + 1024)) == write(fn, c=pool(vs=A[10] + 64)) == sg.ERR_ALIAS
    # pages of keys and values that alternate, and that meet
    assert write(fn, c=pool(v=A[10] + 1024, strides=(4096, 4096, 32, 32))) == sg.ERR_ALIAS


def test_read_refusals(fn):
    assert read(fn, N=-1) == sg.ERR_BAD_DIM and read(fn, type_=5) == sg.ERR_BAD_ARG
    assert read(fn, slots=None) == read(fn, k=heads(0, 2)) == sg.ERR_NULL_PTR
    assert read(fn, k=heads(A[2], 3)) == sg.ERR_BAD_DIM
    assert read(fn, k=heads(A[2], 2, ld=100)) == sg.ERR_BAD_LD
    assert read(fn, k=heads(A[4], 2)) == read(fn, v=heads(A[10], 2)) == read(fn, slots=A[2]) == sg.ERR_ALIAS
    assert read(fn, N=0, slots=None) == sg.OK and read(fn, k=None, v=None) == sg.OK


def test_attend_refusals(fn):
    assert attend(fn, B=-1) == attend(fn, B=(1 << 30) + 1) == attend(fn, pages=-1) == sg.ERR_BAD_DIM
    assert attend(fn, pages=1 << 28, ldt=1 << 28) == sg.ERR_BAD_DIM
    # strips of 16 tokens are counted in 32 bits: 4 heads of 2^15 sequences of 2^18 tokens
    assert attend(fn, B=1 << 15, pages=1 << 14, ldt=1 << 14) == sg.ERR_TOO_LARGE
    assert attend(fn, type_=2) == attend(fn, scale=NAN) == attend(fn, scale=INF) == attend(fn, window=-1) == sg.ERR_BAD_ARG
    for name in ("q", "out", "table", "lens", "c"):
        assert attend(fn, **{name: None}) == sg.ERR_NULL_PTR
    assert attend(fn, q=heads(A[0], 3), out=heads(A[1], 3)) == attend(fn, out=heads(A[1], 2)) == sg.ERR_BAD_DIM
    assert attend(fn, ldt=7) == attend(fn, out=heads(A[1], 4, ld=200)) == sg.ERR_BAD_LD
    assert attend(fn, table=A[5] + 2) == attend(fn, lens=A[6] + 1) == attend(fn, lse=A[7] + 2) == sg.ERR_BAD_ARG
    for place in (A[0], A[5], A[6], A[7], A[10], A[13]):
        assert attend(fn, out=heads(place, 4)) == sg.ERR_ALIAS
    for place in (A[0], A[5], A[6], A[11], A[12]):
        assert attend(fn, lse=place) == sg.ERR_ALIAS
    assert attend(fn, B=0, q=None, out=None, lens=None) == sg.OK


def test_status_string(fn):
    assert sg.status_string(sg.ERR_BAD_INDEX) not in ("unknown status", sg.status_string(sg.ERR_BAD_ARG))
