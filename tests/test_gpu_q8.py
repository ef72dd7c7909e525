"""The 8-bit serving operators against their 64-bit definitions (see q8_ref):
quantised rows, RMS norm with quantisation, the 8-bit linear product and the
expert layer, over lengths from one up, odd sizes, strides and offsets, rows of
zeros, NaN, infinities and extreme values, streams and graph capture.

Tolerances.  A result in bf16 may lie half a unit in the last place (2^-8
relative) from the definition, besides its FP32 error.  FP32 errors: a linear
element takes at most four roundings before the activation (whose slope is
below 1.13) and six within it, CUDA's tanhf and expf counted as two units in
the last place each: below 16 * 2^-24 = 2^-20 of |product| + |bias|.  A row's
scale takes a sum of squares (at most 42 additions deep, half of whose error
reaches the root) and five more roundings: below 32 * 2^-24 < 2e-6.
"""

import numpy as np
import pytest

import q8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402

BF16_HALF = 2.0 ** -8
ROW_TOL, LINEAR_TOL = 2e-6, 2.0 ** -20
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


def to_type(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DT[dt])


def f32(t):
    return t.float().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, tol, dt="fp32"):
    """Within `tol` (an array), plus the output type's rounding; NaN and
    infinities where the definition has them."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    limit = tol + (BF16_HALF * (1 + 2.0 ** -6) * np.abs(want) if dt == "bf16" else 0.0) + 2.0 ** -140
    off = np.abs(got - want)
    bad = fine & (off > limit)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {np.nanmax(np.where(fine, off / limit, 0)):.2f}x the bound"


# ---- rows ------------------------------------------------------------------

def rows_reference(x, residual, weight, eps):
    h32 = f32(x) if residual is None else f32(x) + f32(residual)
    if weight is None:
        q, step = ref.quantize(h32)
        return h32, q, step, None
    with np.errstate(over="ignore", invalid="ignore"):
        p = h32 * weight[None]
    q, step = ref.quantize(p)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        r = 1.0 / np.sqrt((h32.astype(np.float64) ** 2).mean(1) + eps)
        scale = np.where(step == 0, 0.0, step * r)
        y = p.astype(np.float64) * r[:, None]
    return h32, q, scale, y


def run_rows(x, residual=None, weight=None, eps=1e-6, dt="fp32", with_h=False, with_y=False, pad=0,
             offset=0, in_place=None):
    M, K = x.shape
    px = ref.Padded(to_type(x, dt), K + pad, offset)
    pr = None if residual is None else ref.Padded(to_type(residual, dt), K + 2 * pad, offset)
    blank = torch.zeros((M, K), dtype=DT[dt])
    ph = ref.Padded(blank, K + pad, offset) if with_h else None
    if in_place:
        ph = px if in_place == "x" else pr
    py = ref.Padded(blank, K + pad, offset) if with_y else None
    pq = ref.Padded(torch.zeros((M, K), dtype=torch.int8), K + pad, offset)
    scale = torch.full((M,), 7.0, device="cuda")
    want = rows_reference(px.view, None if pr is None else pr.view, weight, eps)
    if weight is None:
        sg.quantize_q8(px.view, pq.view, scale)
    else:
        sg.rmsnorm_q8(px.view, torch.from_numpy(weight).cuda(), pq.view, scale,
                      residual=None if pr is None else pr.view, h=None if ph is None else ph.view,
                      y=None if py is None else py.view, eps=eps)
    assert sg.status() == sg.OK
    for p in (px, pr, ph, py, pq):
        assert p is None or p.outside_intact(), "a write landed outside its array"
    for p in (px, pr):
        assert p is None or p is ph or p.unchanged(), "an input was modified"
    h32, q, step, y = want
    assert np.array_equal(pq.view.cpu().numpy().astype(np.int64), q)
    close(scale, step, ROW_TOL * np.abs(np.nan_to_num(step)))
    if ph is not None:
        exact = ref.bf16_round(h32) if dt == "bf16" else h32.astype(np.float64)
        assert np.array_equal(f64(ph.view), exact, equal_nan=True)
    if py is not None:
        close(py.view, y, ROW_TOL * np.abs(np.nan_to_num(y)), dt)
    return pq.view.cpu(), scale.cpu()


def sample(rng, M, K):
    x = rng.standard_normal((M, K))
    x[:, :: max(1, K // 5)] *= 8.0
    return x.astype(np.float32)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 2), (1, 31), (5, 32), (2, 255), (4, 1000), (3, 4092), (7, 4096),
                                 (2, 4100), (3, 5555), (2, 8191), (2, 8200), (1, 14336), (2, 16384), (2, 16400),
                                 (1, 16391), (1, 40000)])
def test_rows(M, K, dt):
    rng = np.random.default_rng(M * 100003 + K)
    x, r = sample(rng, M, K), 2 * sample(rng, M, K)
    w = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    run_rows(x, dt=dt)
    run_rows(x, r, w, dt=dt, with_h=True, with_y=True)
    run_rows(x, None, w, dt=dt)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (4, 4), (8, 8), (16, 0), (4, 0), (0, 2)])
def test_rows_strides_and_offsets(pad, offset, dt):
    rng = np.random.default_rng(pad * 10 + offset)
    M, K = 5, 512
    w = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    run_rows(sample(rng, M, K), sample(rng, M, K), w, dt=dt, with_h=True, with_y=True, pad=pad, offset=offset)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("K", [64, 1001, 4096, 20000])
def test_rows_in_place(which, K):
    rng = np.random.default_rng(K)
    w = np.ones(K, dtype=np.float32)
    run_rows(sample(rng, 3, K), sample(rng, 3, K), w, dt="bf16", with_y=True, in_place=which)


@pytest.mark.parametrize("K", [40, 515, 4096, 17000])
@pytest.mark.parametrize("norm", [False, True])
def test_rows_of_extreme_values(K, norm):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((12, K)).astype(np.float32)
    x[0] = 0.0
    x[1, K // 2] = np.nan
    x[2, K - 1] = np.inf
    x[3, 0] = -np.inf
    x[4] *= 1e-42                       # below the smallest normal number
    x[5] *= 1e-37
    x[6] *= 3e36                        # squares overflow FP32
    x[7] = 0.0
    x[7, K - 1] = 1e-45                 # the smallest number
    x[8] = 3.4028235e38                 # the largest, everywhere
    x[9] = -1.0
    x[10, :] = 0.0
    x[10, 0] = -5.0
    w = np.ones(K, dtype=np.float32) if norm else None
    run_rows(x, None, w, with_y=norm)
    if norm:
        run_rows(x, None, w, eps=0.0)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("K", [33, 520, 1000, 1028, 2056, 4092, 4100, 5002, 8184, 16384, 16390])
def test_many_rows(K, dt):
    """More rows than two an SM, where a thread takes several vectors; some rows are
    of extreme values."""
    rng = np.random.default_rng(K)
    M = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    x, r = sample(rng, M, K), sample(rng, M, K)
    x[5, K // 2], x[6, K - 1], x[7, 0] = np.nan, np.inf, -np.inf
    x[8, :], r[8, :] = 0.0, 0.0
    x[9] *= 1e-30
    r[9] = 0.0
    w = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    run_rows(x, dt=dt)
    run_rows(x, r, w, dt=dt, with_h=True, with_y=True)
    run_rows(x, None, w, dt=dt)


def test_rows_norm_nan_weight_marks_the_row():
    w = np.ones(64, dtype=np.float32)
    w[3] = np.nan
    q, s = run_rows(np.ones((2, 64), dtype=np.float32), None, w)
    assert torch.isnan(s).all() and (q == 0).all()


def test_rows_empty():
    q = torch.zeros((0, 8), dtype=torch.int8, device="cuda")
    sg.quantize_q8(torch.zeros((0, 8), device="cuda"), q, torch.zeros(0, device="cuda"))
    s = torch.full((3,), 5.0, device="cuda")
    sg.quantize_q8(torch.zeros((3, 0), device="cuda"), torch.zeros((3, 0), dtype=torch.int8, device="cuda"), s)
    assert (s.cpu() == 0).all()
    s.fill_(5.0)
    sg.rmsnorm_q8(torch.zeros((3, 0), device="cuda"), torch.zeros(0, device="cuda"),
                  torch.zeros((3, 0), dtype=torch.int8, device="cuda"), s)
    assert (s.cpu() == 0).all()
    assert sg.status() == sg.OK


# ---- linear ----------------------------------------------------------------

def run_linear(M, N, K, dt="fp32", bias=False, act="none", pads=(0, 0, 0), offsets=(0, 0, 0), seed=0,
               extremes=False, xs=None):
    rng = np.random.default_rng(seed + M * 7 + N * 11 + K * 13)
    if extremes:
        xq = rng.choice(np.array([-128, 127], dtype=np.int8), (M, K))
        wq = rng.choice(np.array([-128, 127], dtype=np.int8), (N, K))
        xq[0], wq[0] = -128, -128            # the largest sum there is
        if M > 1:
            xq[1] = 127
    else:
        xq = np.clip(np.rint(32 * rng.standard_normal((M, K))), -127, 127).astype(np.int8)
        wq = np.clip(np.rint(32 * rng.standard_normal((N, K))), -127, 127).astype(np.int8)
    xs = (rng.uniform(0.5, 1.5, M) / 32).astype(np.float32) if xs is None else xs
    ws = (rng.uniform(0.5, 1.5, N) / (32 * max(K, 1) ** 0.5)).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    px, pw = ref.Padded(xq, max(K, 1) + pads[0], offsets[0]), ref.Padded(wq, max(K, 1) + pads[1], offsets[1])
    pc = ref.Padded(torch.full((M, N), 3.0, dtype=DT[dt]), max(N, 1) + pads[2], offsets[2])
    sg.linear_q8(px.view, torch.from_numpy(xs).cuda(), pw.view, torch.from_numpy(ws).cuda(), pc.view,
                 bias=None if b is None else torch.from_numpy(b).cuda(), activation=act)
    assert sg.status() == sg.OK
    assert pc.outside_intact() and px.unchanged() and pw.unchanged()
    want, size = ref.linear(xq, xs, wq, ws, b, act)
    # past 2^24 a sum is rounded once for every 1024 k
    tol = (LINEAR_TOL + (K // 1024) * 2.0 ** -24 * (1 if not extremes else 4)) * np.nan_to_num(size)
    close(pc.view, want, tol, dt)
    return pc.view


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 17, 3), (2, 100, 64), (3, 33, 65), (7, 129, 130), (8, 256, 512), (9, 255, 513), (16, 300, 1000),
    (1, 512, 4096), (16, 130, 4096), (17, 64, 256), (31, 200, 96), (33, 257, 1024), (64, 128, 1040), (65, 384, 2048),
    (100, 500, 200), (128, 130, 1025), (129, 129, 129), (200, 640, 4096), (256, 256, 64), (257, 513, 1100),
    (300, 1000, 48), (520, 260, 3000), (1, 40, 14336), (40, 24, 14336), (700, 16, 272),
    # enough blocks of 16 tokens x 32 channels that the tensor-core tiles take over
    (40, 4100, 256), (70, 4096, 528), (130, 2500, 1040), (200, 2300, 96), (300, 1100, 2080), (513, 700, 80),
    (260, 1300, 4096), (1030, 300, 144), (18, 9800, 64)])
def test_linear(M, N, K, dt):
    run_linear(M, N, K, dt)


@pytest.mark.parametrize("M", [1, 8, 16, 24, 48, 130, 300, 1100])
@pytest.mark.parametrize("pads,offsets", [
    ((1, 0, 0), (0, 0, 0)), ((0, 1, 0), (0, 0, 0)), ((0, 0, 1), (0, 0, 1)), ((0, 0, 0), (1, 0, 0)),
    ((0, 0, 0), (0, 3, 0)), ((16, 16, 8), (16, 32, 8)), ((4, 8, 4), (4, 8, 4)), ((5, 7, 3), (2, 9, 5))])
def test_linear_strides_and_offsets(M, pads, offsets):
    run_linear(M, 144, 272, "bf16", True, "none", pads, offsets)


@pytest.mark.parametrize("M,N", [(1, 200), (16, 200), (40, 200), (128, 200), (20, 8000), (40, 4500), (128, 2000),
                                 (280, 1200)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("bias", [False, True])
def test_linear_epilogue(M, N, act, bias):
    run_linear(M, N, 320, "fp32", bias, act)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M,N", [(3, 200), (40, 200), (40, 4500), (280, 1200)])
def test_linear_bf16_activations_of_large_values(M, N, act):
    """Both tails and beyond: products from 0 to about 200 in size.  A fast
    exponential is off by (2 + 1.2 |x|) units in the last place, of a value that is
    negligible or 1 where |x| is large: below 2^-17 of the result."""
    rng = np.random.default_rng(M)
    K = 96
    xq, wq = (rng.integers(-127, 128, (n, K)).astype(np.int8) for n in (M, N))
    xs = (10.0 ** rng.uniform(-4, 0.5, M) / 127).astype(np.float32)
    ws = (np.ones(N) * 60 / (127 * K ** 0.5)).astype(np.float32)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    sg.linear_q8(*[torch.from_numpy(a).cuda() for a in (xq, xs, wq, ws)], out, activation=act)
    want, size = ref.linear(xq, xs, wq, ws, None, act)
    close(out, want, LINEAR_TOL * size + 2.0 ** -17 * np.abs(want), "bf16")


@pytest.mark.parametrize("M,N,K", [(1, 40, 1024), (5, 40, 4096), (16, 20, 20000), (33, 40, 1024), (70, 130, 4096),
                                   (300, 140, 8192), (20, 130, 131071), (70, 2600, 4096), (40, 5000, 1024),
                                   (300, 1100, 2048), (1040, 260, 5000)])
def test_linear_extreme_values(M, N, K):
    run_linear(M, N, K, extremes=True)


@pytest.mark.parametrize("M,N", [(1, 70), (3, 70), (12, 70), (40, 70), (260, 70), (40, 4900), (100, 2600), (270, 1100)])
def test_linear_exact_sums(M, N):
    """Sums below 2^24 are whole numbers: scales of one give them exactly."""
    rng = np.random.default_rng(M)
    K = 5000
    xq, wq = (rng.integers(-60, 61, (n, K)).astype(np.int8) for n in (M, N))
    out = torch.empty((M, N), device="cuda")
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    sg.linear_q8(torch.from_numpy(xq).cuda(), one(M), torch.from_numpy(wq).cuda(), one(N), out)
    want = xq.astype(np.int64) @ wq.astype(np.int64).T
    assert np.abs(want).max() < 2 ** 24
    assert np.array_equal(out.cpu().numpy().astype(np.int64), want)


@pytest.mark.parametrize("M,N", [(3, 70), (20, 70), (150, 70), (40, 4900), (150, 2400), (300, 1100)])
def test_linear_nan_scale_stays_in_its_row(M, N):
    xs = np.full(M, 0.02, dtype=np.float32)
    xs[1] = np.nan
    out = run_linear(M, N, 96, xs=xs)
    assert torch.isnan(out[1]).all() and not torch.isnan(out[0]).any() and not torch.isnan(out[2:]).any()


@pytest.mark.parametrize("M", [2, 50])
def test_linear_without_terms(M):
    run_linear(M, 30, 0, "fp32", True, "relu")
    run_linear(0, 30, 16)
    run_linear(M, 0, 16)


# ---- expert layer ------------------------------------------------------------

def make_moe(T, E, H, inner, dt, seed=0, same=False):
    rng = np.random.default_rng(seed + T + 31 * E + 7 * H + inner)
    x = f32(to_type(rng.standard_normal((1 if same else T, H)), dt))
    if same:
        x = np.repeat(x, T, 0)
    router = (rng.standard_normal((E, H)) / H ** 0.5).astype(np.float32)
    w_up = np.clip(np.rint(32 * rng.standard_normal((E, 2 * inner, H))), -127, 127).astype(np.int8)
    w_down = np.clip(np.rint(32 * rng.standard_normal((E, H, inner))), -127, 127).astype(np.int8)
    s_up = (rng.uniform(0.5, 1.5, (E, 2 * inner)) / (32 * H ** 0.5)).astype(np.float32)
    s_down = (rng.uniform(0.5, 1.5, (E, H)) / (32 * inner ** 0.5)).astype(np.float32)
    return x, router, w_up, s_up, w_down, s_down


def cuda(a, offset=0):
    """A contiguous device copy, `offset` elements into its buffer."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v


def call_moe(args, k, dt, renorm=True, pad=0, offset=0, stream=None, routing=True):
    x, router, w_up, s_up, w_down, s_down = args
    T, H = x.shape
    px = ref.Padded(to_type(x, dt), H + pad, offset)
    po = ref.Padded(torch.zeros((T, H), dtype=DT[dt]), H + 2 * pad, offset)
    pr = ref.Padded(router, H + pad, offset)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda") if routing else None
    gates = torch.zeros((T, k), device="cuda") if routing else None
    sg.moe_q8(px.view, pr.view, cuda(w_up, offset), cuda(s_up), cuda(w_down, offset), cuda(s_down), po.view, k,
              renormalize=renorm, ids=ids, gates=gates, stream=stream)
    assert sg.status(stream) == sg.OK
    assert po.outside_intact() and px.unchanged() and pr.unchanged()
    return po.view, ids, gates


def check_moe(args, k, dt, renorm=True, **kw):
    out, ids, gates = call_moe(args, k, dt, renorm, **kw)
    want, slack, wids, wgates, gap = ref.moe(*args, k, renorm)
    assert gap > 1e-5, "inputs with near ties have no defined choice"
    assert np.array_equal(ids.cpu().numpy(), wids)
    # a logit's sum is at most H/256 + 13 additions deep, terms of about 1/sqrt(H): far below 1e-5
    close(gates, wgates, 2e-5 * np.abs(wgates))
    close(out, want, slack + 2e-5 * np.abs(want), dt)
    return out


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,k,H,inner", [
    (1, 1, 1, 16, 16), (1, 4, 2, 64, 32), (2, 3, 3, 33, 17), (5, 8, 2, 128, 100), (8, 8, 2, 256, 96),
    (16, 64, 6, 128, 64), (17, 4, 2, 130, 70), (33, 5, 2, 64, 48), (64, 4, 1, 96, 80), (64, 40, 16, 48, 24),
    (3, 130, 4, 1024, 40), (2, 512, 8, 64, 16), (4, 8, 2, 2048, 1031), (1, 8, 2, 1500, 2100), (9, 2, 1, 515, 300)])
def test_moe(T, E, k, H, inner, dt):
    check_moe(make_moe(T, E, H, inner, dt), k, dt, renorm=(T + k) % 2 == 0)


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 2), (16, 16)])
def test_moe_strides_and_offsets(pad, offset):
    check_moe(make_moe(5, 6, 144, 80, "bf16"), 2, "bf16", pad=pad, offset=offset)


@pytest.mark.parametrize("T", [7, 16, 40])
def test_moe_one_expert_takes_every_token(T):
    out = check_moe(make_moe(T, 6, 96, 64, "fp32", same=True), 2, "fp32")
    assert bool((out == out[0]).all())


def test_moe_ties_go_to_the_lowest_index():
    x, router, *rest = make_moe(4, 10, 64, 32, "fp32")
    router[:] = router[3]               # every logit of a token is the same number
    _, ids, gates = call_moe((x, router, *rest), 4, "fp32")
    assert np.array_equal(ids.cpu().numpy(), np.tile(np.arange(4), (4, 1)))
    assert np.allclose(gates.cpu().numpy(), 0.25, rtol=1e-6)
    router[:] = 0.0
    router[7] = -0.0
    _, ids, _ = call_moe((x, router, *rest), 2, "fp32")
    assert np.array_equal(ids.cpu().numpy(), np.tile(np.arange(2), (4, 1)))


def test_moe_nan_and_infinite_tokens_stay_in_their_rows():
    args = make_moe(6, 8, 64, 32, "fp32")
    clean, ids0, _ = call_moe(args, 2, "fp32")
    x = args[0].copy()
    x[1, 5] = np.nan
    x[4, 0] = np.inf
    out, ids, _ = call_moe((x, *args[1:]), 2, "fp32")
    fine = [0, 2, 3, 5]
    assert torch.isnan(out[1]).all() and torch.isnan(out[4]).all()
    assert torch.equal(out[fine], clean[fine]) and torch.equal(ids[fine], ids0[fine])
    got = ids.cpu().numpy()
    assert ((0 <= got) & (got < 8)).all() and all(len(set(r)) == 2 for r in got)


def test_moe_zero_token():
    args = make_moe(3, 4, 64, 32, "bf16")
    args[0][1] = 0.0
    out, _, _ = call_moe(args, 2, "bf16")
    assert (out[1] == 0).all() and torch.isfinite(out).all()


def test_moe_is_its_parts():
    """One token's row is the composition of the other operators, weighted."""
    T, E, H, inner, k = 4, 5, 256, 96, 2
    x, router, w_up, s_up, w_down, s_down = make_moe(T, E, H, inner, "fp32")
    out, ids, gates = call_moe((x, router, w_up, s_up, w_down, s_down), k, "fp32")
    dx = torch.from_numpy(x).cuda()
    xq, xs = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    sg.quantize_q8(dx, xq, xs)
    want = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            up = torch.empty((1, 2 * inner), device="cuda")
            sg.linear_q8(xq[t:t + 1], xs[t:t + 1], cuda(w_up[e]), cuda(s_up[e]), up)
            g, u = up[:, :inner], up[:, inner:]
            hid = (g / (1 + torch.exp(-g)) * u).contiguous()
            hq, hs = torch.empty((1, inner), dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
            sg.quantize_q8(hid, hq, hs)
            down = torch.empty((1, H), device="cuda")
            sg.linear_q8(hq, hs, cuda(w_down[e]), cuda(s_down[e]), down)
            want[t] += float(gates[t, j]) * down[0].double().cpu()
    want = want.numpy()
    # the same whole numbers throughout but for torch's exp, which may move a hidden value by a step
    _, slack, *_ = ref.moe(x, router, w_up, s_up, w_down, s_down, k, True)
    close(out, want, slack + 2e-5 * np.abs(want))


def test_moe_without_tokens():
    x, *rest = make_moe(1, 4, 64, 32, "fp32")
    sg.moe_q8(torch.zeros((0, 64), device="cuda"), *[cuda(a) for a in rest], torch.zeros((0, 64), device="cuda"), 2)
    assert sg.status() == sg.OK


# ---- shared conduct ------------------------------------------------------------

def chain(stream=None, M=5, H=256, inner=192, seed=3, wide=0):
    """norm -> up -> quantise -> down on fixed inputs, then the expert layer."""
    rng = np.random.default_rng(seed)
    dev = {}
    dev["x"] = to_type(rng.standard_normal((M, H)), "bf16").cuda()
    dev["r"] = to_type(rng.standard_normal((M, H)), "bf16").cuda()
    dev["w"] = torch.ones(H, device="cuda")
    moe = [cuda(a) for a in make_moe(M, 6, H, inner, "bf16")[1:]]
    up, sup = moe[1][0], moe[2][0]
    dn, sdn = moe[3][0], moe[4][0]
    b = {"h": torch.empty_like(dev["x"]), "y": torch.empty_like(dev["x"]),
         "q": torch.empty((M, H), dtype=torch.int8, device="cuda"), "s": torch.empty(M, device="cuda"),
         "hid": torch.empty((M, 2 * inner), dtype=torch.bfloat16, device="cuda"),
         "hq": torch.empty((M, inner), dtype=torch.int8, device="cuda"), "hs": torch.empty(M, device="cuda"),
         "o": torch.empty((M, H), dtype=torch.bfloat16, device="cuda"),
         "m": torch.empty((M, H), dtype=torch.bfloat16, device="cuda")}
    if wide:
        dev["ww"] = cuda(rng.integers(-127, 128, (wide, H)).astype(np.int8))
        dev["sw"] = torch.full((wide,), 1e-3, device="cuda")
        b["wide"] = torch.empty((M, wide), device="cuda")

    def go():
        sg.rmsnorm_q8(dev["x"], dev["w"], b["q"], b["s"], residual=dev["r"], h=b["h"], y=b["y"], stream=stream)
        sg.linear_q8(b["q"], b["s"], up, sup, b["hid"], activation="silu", stream=stream)
        sg.quantize_q8(b["hid"][:, :inner], b["hq"], b["hs"], stream=stream)
        sg.linear_q8(b["hq"], b["hs"], dn, sdn, b["o"], stream=stream)
        if wide:        # enough output for the tensor-core tiles
            sg.linear_q8(b["q"], b["s"], dev["ww"], dev["sw"], b["wide"], stream=stream)
        sg.moe_q8(b["y"], *moe, b["m"], 2, stream=stream)
    return go, b


@pytest.mark.parametrize("M,wide", [(1, 0), (16, 0), (50, 3500), (60, 9000)])
def test_repeats_are_the_same_bits(M, wide):
    go, b = chain(M=M, wide=wide)
    go()
    first = {n: t.clone() for n, t in b.items()}
    for _ in range(3):
        go()
    assert sg.status() == sg.OK
    assert all(torch.equal(first[n], t) for n, t in b.items())


@pytest.mark.parametrize("M,wide", [(2, 0), (40, 4500)])
def test_side_stream_and_graph(M, wide):
    go, b = chain(M=M, wide=wide)
    go()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in b.items()}
    side = torch.cuda.Stream()
    go2, b2 = chain(stream=side, M=M, wide=wide)
    side.wait_stream(torch.cuda.current_stream())
    go2()
    assert sg.status(side) == sg.OK
    assert all(torch.equal(want[n], t) for n, t in b2.items())
    for t in b2.values():
        t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go2()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert sg.status() == sg.OK
    assert all(torch.equal(want[n], t) for n, t in b2.items())


def test_two_streams_at_once():
    """Calls of two streams overlap on the GPU and keep apart."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [chain(stream=s, M=40, seed=5 + i, wide=4500) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for go, _ in runs:
        go()
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in b.items()} for _, b in runs]
    for _ in range(20):
        for go, _ in runs:
            go()
    torch.cuda.synchronize()
    for s in streams:
        assert sg.status(s) == sg.OK
    assert all(torch.equal(w[n], t) for w, (_, b) in zip(want, runs) for n, t in b.items())


def test_refused_calls_change_nothing():
    x = torch.randn((4, 64), device="cuda")
    q = torch.full((4, 64), 9, dtype=torch.int8, device="cuda")
    s = torch.full((4,), 9.0, device="cuda")
    for bad in (lambda: sg.quantize_q8(x.double(), q, s), lambda: sg.quantize_q8(x, q.to(torch.uint8), s),
                lambda: sg.quantize_q8(x.cpu(), q, s), lambda: sg.quantize_q8(x, q, s.cpu()),
                lambda: sg.linear_q8(q, s, q, s, x.half()[:, :4]),
                lambda: sg.rmsnorm_q8(x, torch.ones(64, device="cuda"), q, s, residual=x.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sg.quantize_q8(x, q[:, :32], s), lambda: sg.quantize_q8(x.t(), q.t(), s),
                lambda: sg.quantize_q8(x, q, s[:3]), lambda: sg.linear_q8(q, s, q[:, :32], s, x[:, :4]),
                lambda: sg.linear_q8(q, s, q, s, x[:, :4], activation="tanh"),
                lambda: sg.linear_q8(q, s, q, s, x[:, :5])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sg.SgemmError) as e:      # the output takes an input's place
        sg.rmsnorm_q8(x, torch.ones(64, device="cuda"), q, s, y=x)
    assert e.value.code == sg.ERR_ALIAS
    with pytest.raises(sg.SgemmError) as e:
        sg.rmsnorm_q8(x, torch.ones(64, device="cuda"), q, s, eps=-1.0)
    assert e.value.code == sg.ERR_BAD_ARG
    args = [cuda(a) for a in make_moe(4, 4, 64, 32, "fp32")]
    out = torch.full((4, 64), 9.0, device="cuda")
    for k in (0, 5):
        with pytest.raises(sg.SgemmError) as e:
            sg.moe_q8(*args, out, k)
        assert e.value.code == sg.ERR_BAD_DIM
    big = torch.zeros((65, 64), device="cuda")
    with pytest.raises(sg.SgemmError) as e:
        sg.moe_q8(big, *args[1:], torch.zeros_like(big), 2)
    assert e.value.code == sg.ERR_TOO_LARGE
    torch.cuda.synchronize()
    assert (q == 9).all() and (s == 9).all() and (out == 9).all()
    assert sg.status() == sg.OK
