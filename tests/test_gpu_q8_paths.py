"""The 8-bit operators on sizes that reach every form of their kernels: the
256-token tile of the linear product, expert units of several row tiles and
several stages, 1 to 16 tokens to an expert, and the rows that a warp takes.

Each test restates the rule that leads a call to its form and checks that its
sizes meet it.  Definitions and tolerances are those of test_gpu_q8.
"""

import numpy as np
import pytest

import q8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402
from test_gpu_q8 import check_moe, run_linear, run_rows, sample, to_type  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def up(n, d):
    return -(-n // d)


# ---- linear: tiles of 256 tokens ---------------------------------------------------

def wide_tile(M, N):
    """More than 128 tokens, and tiles of 256 x 256 for at least a quarter of the SMs."""
    return M > 128 and up(N, 256) * up(M, 256) >= sms() // 4


# remainders of every kind inside the last tiles, one chunk of 1024 k and several, and
# (2100 x 4000) more tiles than pairs of SMs
WIDE = [(1001, 4092, 1100), (513, 3600, 80), (300, 5200, 2100), (1030, 2100, 1024), (2100, 4000, 2300)]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", WIDE)
def test_wide_tiles(M, N, K, dt):
    assert wide_tile(M, N)
    run_linear(M, N, K, dt)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_wide_tiles_epilogue(act, dt):
    assert wide_tile(700, 3300)
    run_linear(700, 3300, 320, dt, True, act)


@pytest.mark.parametrize("pads,offsets", [
    ((1, 0, 0), (0, 0, 0)), ((0, 1, 0), (0, 0, 0)), ((0, 0, 1), (0, 0, 1)), ((0, 0, 0), (0, 3, 0)),
    ((5, 7, 3), (2, 9, 5))])
def test_wide_tiles_strides_and_offsets(pads, offsets):
    assert wide_tile(600, 3400)
    run_linear(600, 3400, 1296, "bf16", True, "none", pads, offsets)


@pytest.mark.parametrize("M,N,K", [(520, 3600, 3000), (2070, 2300, 1040)])
def test_wide_tiles_extreme_values(M, N, K):
    assert wide_tile(M, N)
    run_linear(M, N, K, extremes=True)


def test_wide_tiles_exact_sums():
    M, N, K = 530, 3700, 5000
    assert wide_tile(M, N)
    rng = np.random.default_rng(1)
    xq, wq = (rng.integers(-60, 61, (n, K)).astype(np.int8) for n in (M, N))
    out = torch.empty((M, N), device="cuda")
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    sg.linear_q8(torch.from_numpy(xq).cuda(), one(M), torch.from_numpy(wq).cuda(), one(N), out)
    # whole numbers below 2^53: float64 gives them exactly
    want = xq.astype(np.float64) @ wq.astype(np.float64).T
    assert np.abs(want).max() < 2 ** 24
    assert np.array_equal(out.cpu().numpy().astype(np.float64), want)


# ---- expert layer --------------------------------------------------------------

class Division:
    """How the expert kernel divides one projection (rows of K values, `rows`
    results, `per_tile` of them to a row tile) over `chunks` groups of tokens."""

    def __init__(self, K, rows, per_tile, chunks):
        steps, shift = up(K, 64), K % 16 != 0
        self.rt = 4 if steps <= 8 else 2 if steps <= 16 else 1
        kb = 8 // self.rt * 4
        blocks = (K - 15) // 64 if shift else K // 64
        self.stages = max(1, up(blocks, kb))
        tiles = up(rows, per_tile * self.rt)
        self.sub = {1: 4, 2: 2, 4: 1}[self.rt]
        while self.sub > 1 and tiles * chunks < 6 * self.sub * sms():
            self.sub //= 2


def make_moe(T, E, H, inner, dt, seed=0):
    rng = np.random.default_rng(seed + T + 31 * E + 7 * H + inner)
    x = to_type(rng.standard_normal((T, H)), dt).float().numpy()
    router = (rng.standard_normal((E, H)) / H ** 0.5).astype(np.float32)
    w_up = rng.integers(-100, 101, (E, 2 * inner, H), dtype=np.int8)
    w_down = rng.integers(-100, 101, (E, H, inner), dtype=np.int8)
    s_up = (rng.uniform(0.5, 1.5, (E, 2 * inner)) / (58 * H ** 0.5)).astype(np.float32)
    s_down = (rng.uniform(0.5, 1.5, (E, H)) / (58 * inner ** 0.5)).astype(np.float32)
    return x, router, w_up, s_up, w_down, s_down


def chunks_of(x, router, k):
    """Groups of up to 16 tokens of one expert, over all experts."""
    logits = x.astype(np.float64) @ router.astype(np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    counts = np.bincount(ids.ravel(), minlength=router.shape[0])
    return int(sum(up(c, 16) for c in counts))


# T, E, k, H, I, dt, then what the case is for: tiles to a unit and stages to a tile, gate/up and down
CASES = [
    (1, 2, 2, 2304, 7424, "bf16", (2, 1), (2, 4)),         # one token, units of two tiles, several stages
    (16, 64, 8, 1088, 1088, "bf16", (4, 4), (1, 1)),       # units of four tiles in both projections
    (64, 128, 16, 576, 576, "fp32", (2, 2), (1, 1)),       # units of two tiles of two; 2 to 16 tokens to an expert
    (3, 4, 4, 2304, 3712, "fp32", (2, 1), (2, 2)),         # dp4a with 3 tokens, both loops
    (8, 4, 4, 2304, 3712, "bf16", (2, 1), (2, 2)),         # one block of tokens by MMA
    (16, 4, 4, 2304, 3712, "bf16", (2, 1), (2, 2)),        # two blocks
    (12, 2, 1, 2500, 2700, "bf16", (1, 1), (2, 2)),        # rows that are no multiple of 16 bytes
    (2, 4, 4, 2309, 3721, "fp32", (2, 1), (2, 2)),         # the same, units of two tiles
]


@pytest.mark.parametrize("T,E,k,H,inner,dt,sub,stages", CASES)
def test_units_of_several_tiles_and_stages(T, E, k, H, inner, dt, sub, stages):
    args = make_moe(T, E, H, inner, dt)
    chunks = chunks_of(args[0], args[1], k)
    gate_up, down = Division(H, inner, 8, chunks), Division(inner, H, 16, chunks)
    if sms() == 152:
        assert (gate_up.sub, down.sub) == sub
    assert (gate_up.stages, down.stages) == stages
    check_moe(args, k, dt, renorm=T % 2 == 0)


@pytest.mark.parametrize("H,inner", [(2304, 2240), (2309, 2251)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 17, 40])
def test_tokens_of_one_expert_over_several_stages(T, H, inner):
    assert Division(H, inner, 8, 1).stages > 1 and Division(inner, H, 16, 1).stages > 1
    check_moe(make_moe(T, 1, H, inner, "bf16"), 1, "bf16")


# ---- rows ------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("K,rows", [(8, 3), (64, 3), (136, 3), (256, 3), (512, 3), (64, 10000)])
def test_rows_of_a_warp(K, rows, dt):
    """Rows of at most 64 vectors of 16 bytes, more than two to an SM (`rows` more; with
    10000 a warp takes several).  512 in FP32 is past that, on the other side of the rule."""
    rng = np.random.default_rng(K)
    M = 2 * sms() + rows
    if rows == 10000:
        assert M > 8 * 8 * sms()
    x, r = sample(rng, M, K), sample(rng, M, K)
    x[5, K // 2], x[6, K - 1], x[7, 0] = np.nan, np.inf, -np.inf
    x[8, :], r[8, :] = 0.0, 0.0
    x[9] *= 1e-30
    r[9] = 0.0
    w = (1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    run_rows(x, dt=dt)
    run_rows(x, r, w, dt=dt, with_h=True, with_y=True)
    run_rows(x, None, w, dt=dt)
    run_rows(x, r, w, dt=dt, with_y=True, in_place="residual")


def test_rows_of_a_warp_of_extreme_values():
    rng = np.random.default_rng(2)
    K, M = 128, 2 * sms() + 40
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[0] *= 1e-42                       # below the smallest normal number
    x[1] *= 1e-37
    x[2] *= 3e36                        # squares overflow FP32
    x[3] = 0.0
    x[3, K - 1] = 1e-45                 # the smallest number
    x[4] = 3.4028235e38                 # the largest, everywhere
    w = np.ones(K, dtype=np.float32)
    run_rows(x, None, w, with_y=True)
    run_rows(x, None, w, eps=0.0)
    run_rows(x)
