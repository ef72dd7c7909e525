"""Argument checks of the 8-bit operators through the C ABI, without a GPU: no
call here is accepted, so none reaches the CUDA runtime (pointers are plain
numbers), except empty ones, which return before it."""

import dense_fp32_matrix_row_gb300 as sg
import pytest

X, R, W, H, Y, Q, S, BIG = (i << 30 for i in range(1, 9))


@pytest.fixture(scope="module")
def fn():
    sg.build()
    from dense_fp32_matrix_row_gb300 import q8
    return lambda name, *a: q8._entry(name)(*a)


def quantize(fn, M=4, K=64, x=X, ldx=64, type_=0, q=Q, ldq=64, s=S):
    return fn("sgemm_q8_quantize", M, K, x, ldx, type_, q, ldq, s, None)


def norm(fn, M=4, K=64, x=X, ldx=64, r=R, ldr=64, type_=0, w=W, eps=1e-6, h=H, ldh=64, y=Y, ldy=64, q=Q, ldq=64,
         s=S):
    return fn("sgemm_q8_rmsnorm", M, K, x, ldx, r, ldr, type_, w, eps, h, ldh, y, ldy, q, ldq, s, None)


def linear(fn, M=4, N=8, K=64, x=X, ldx=64, xs=R, w=W, ldw=64, ws=S, bias=H, act=0, c=Y, ldc=8, type_=0):
    return fn("sgemm_q8_linear", M, N, K, x, ldx, xs, w, ldw, ws, bias, act, c, ldc, type_, None)


def moe(fn, T=2, E=4, k=2, H_=64, I=32, x=X, ldx=64, type_=0, router=R, ldr=64, wu=W, ldu=64, su=S, wd=H, ldd=32,
        sd=Q, renorm=1, out=Y, ldo=64, ids=BIG, gates=9 << 30):
    return fn("sgemm_q8_moe", T, E, k, H_, I, x, ldx, type_, router, ldr, wu, ldu, su, wd, ldd, sd, renorm, out, ldo,
              ids, gates, None)


def test_quantize_refusals(fn):
    assert quantize(fn, M=-1) == sg.ERR_BAD_DIM and quantize(fn, K=-1) == sg.ERR_BAD_DIM
    assert quantize(fn, M=1 << 32) == sg.ERR_BAD_DIM
    assert quantize(fn, M=1 << 30, ldx=1 << 20) == sg.ERR_BAD_DIM
    assert quantize(fn, type_=2) == sg.ERR_BAD_ARG
    assert quantize(fn, ldx=63) == sg.ERR_BAD_LD and quantize(fn, ldq=63) == sg.ERR_BAD_LD
    for a in ("x", "q", "s"):
        assert quantize(fn, **{a: None}) == sg.ERR_NULL_PTR
    assert quantize(fn, x=X + 2) == sg.ERR_BAD_ARG and quantize(fn, x=X + 1, type_=1) == sg.ERR_BAD_ARG
    assert quantize(fn, s=S + 1) == sg.ERR_BAD_ARG
    assert quantize(fn, q=X + 4 * 64 * 4 - 1) == sg.ERR_ALIAS
    assert quantize(fn, s=X) == sg.ERR_ALIAS and quantize(fn, s=Q + 64) == sg.ERR_ALIAS
    assert quantize(fn, M=0, x=None, q=None, s=None) == sg.OK


def test_norm_refusals(fn):
    assert norm(fn, w=None) == sg.ERR_NULL_PTR
    assert norm(fn, eps=-1e-9) == sg.ERR_BAD_ARG and norm(fn, eps=float("nan")) == sg.ERR_BAD_ARG
    for a in ("ldx", "ldr", "ldh", "ldy", "ldq"):
        assert norm(fn, **{a: 63}) == sg.ERR_BAD_LD
    assert norm(fn, y=X) == sg.ERR_ALIAS and norm(fn, y=H) == sg.ERR_ALIAS and norm(fn, q=W) == sg.ERR_ALIAS
    # h in the place of x only with x's own rows
    assert norm(fn, h=X + 4) == sg.ERR_ALIAS
    assert norm(fn, h=X, ldh=80) == sg.ERR_ALIAS
    assert norm(fn, h=R + 64 * 4, ldh=64) == sg.ERR_ALIAS
    assert norm(fn, M=0, w=None) == sg.OK


def test_linear_refusals(fn):
    for a in ("M", "N", "K"):
        assert linear(fn, **{a: -1}) == sg.ERR_BAD_DIM
    assert linear(fn, K=131072, ldx=131072, ldw=131072) == sg.ERR_BAD_DIM
    assert linear(fn, M=1 << 31) == sg.ERR_BAD_DIM
    assert linear(fn, act=4) == sg.ERR_BAD_ARG and linear(fn, type_=-1) == sg.ERR_BAD_ARG
    assert linear(fn, ldx=63) == linear(fn, ldw=63) == linear(fn, ldc=7) == sg.ERR_BAD_LD
    for a in ("x", "xs", "w", "ws", "c"):
        assert linear(fn, **{a: None}) == sg.ERR_NULL_PTR
    for a, v in (("c", Y + 2), ("xs", R + 1), ("ws", S + 2), ("bias", H + 3)):
        assert linear(fn, **{a: v}) == sg.ERR_BAD_ARG
    for a in (X, R, W, S, H):
        assert linear(fn, c=a) == sg.ERR_ALIAS
    assert linear(fn, M=0, c=None) == sg.OK and linear(fn, N=0, c=None) == sg.OK


def test_moe_refusals(fn):
    for a in ({"T": -1}, {"E": 0}, {"k": 0}, {"k": 5}, {"H_": 0}, {"I": 0}, {"H_": 131072}):
        assert moe(fn, **a) == sg.ERR_BAD_DIM
    assert moe(fn, T=65) == moe(fn, E=513) == moe(fn, E=32, k=17) == sg.ERR_TOO_LARGE
    assert moe(fn, type_=7) == sg.ERR_BAD_ARG
    for a in ("ldx", "ldr", "ldu", "ldd", "ldo"):
        assert moe(fn, **{a: 31}) == sg.ERR_BAD_LD
    for a in ("x", "router", "wu", "su", "wd", "sd", "out"):
        assert moe(fn, **{a: None}) == sg.ERR_NULL_PTR
    for a in (X, R, W, S, H, Q, BIG):
        assert moe(fn, out=a) == sg.ERR_ALIAS
    assert moe(fn, out=Y + 2) == moe(fn, gates=(9 << 30) + 2) == sg.ERR_BAD_ARG
    assert moe(fn, T=0, x=None, out=None) == sg.OK
