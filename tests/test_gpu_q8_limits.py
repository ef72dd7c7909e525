"""The 8-bit operators at the ends of their ranges."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402
from test_gpu_q8 import run_rows  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


@pytest.mark.parametrize("M,N", [(1048561, 3), (1100003, 1)])
def test_linear_without_terms_of_many_tokens(M, N):
    """K == 0 gives act(bias) for any number of tokens, beyond 65535 blocks of 16 too."""
    b = torch.tensor([-1.0, 2.0, 0.5][:N], device="cuda")
    out = torch.full((M, N), 9.0, device="cuda")
    sg.linear_q8(torch.empty((M, 0), dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"),
                 torch.empty((N, 0), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"), out, bias=b,
                 activation="relu")
    assert sg.status() == sg.OK
    assert torch.equal(out, torch.relu(b).expand(M, N))


# ---- waits that run out ----------------------------------------------------------

def linear_case(M, N, K):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + N + K)
    xq, wq = (torch.randint(-90, 91, (n, K), generator=gen, device="cuda", dtype=torch.int8) for n in (M, N))
    xs, ws = torch.ones(M, device="cuda"), torch.full((N,), 1e-3, device="cuda")
    out = torch.zeros((M, N), device="cuda")
    return lambda: sg.linear_q8(xq, xs, wq, ws, out), out


def moe_case(T, E, k, H, inner, offset=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + E + H)

    def weights(*shape):
        n = shape[0] * shape[1] * shape[2]
        return torch.randint(-90, 91, (n + offset,), generator=gen, device="cuda",
                             dtype=torch.int8)[offset:].view(shape)

    x, router = (torch.randn(s, generator=gen, device="cuda") for s in ((T, H), (E, H)))
    w_up, w_down = weights(E, 2 * inner, H), weights(E, H, inner)
    s_up, s_down = torch.full((E, 2 * inner), 1e-3, device="cuda"), torch.full((E, H), 1e-3, device="cuda")
    out = torch.zeros((T, H), device="cuda")
    return lambda: sg.moe_q8(x, router, w_up, s_up, w_down, s_down, out, k), out


# the ring by dp4a, 8-bit and FP16 MMAs; tiles of 32, 64, 128 (K whole and divided) and 256 tokens; experts
CASES = {
    "ring 1": lambda: linear_case(1, 9000, 4096), "ring 8": lambda: linear_case(8, 9000, 4096),
    "ring 16": lambda: linear_case(16, 9000, 4096), "tile 32": lambda: linear_case(20, 20000, 1040),
    "tile 64": lambda: linear_case(60, 20000, 4096), "tile 128": lambda: linear_case(128, 20000, 2048),
    "tile 128 divided": lambda: linear_case(100, 4096, 8192), "tile 256": lambda: linear_case(700, 9000, 3000),
    "experts": lambda: moe_case(6, 8, 2, 2048, 1408), "experts, odd rows": lambda: moe_case(6, 8, 2, 1001, 1003),
    "experts, any alignment": lambda: moe_case(6, 8, 2, 512, 1408, offset=3),
}


@pytest.mark.parametrize("name", CASES)
def test_a_wait_that_runs_out_is_reported_and_leaves_nothing_behind(name):
    """With a limit of a nanosecond a wait runs out wherever it finds its event not yet
    there: the kernel records it, lets its copies land and ends.  (The experts' waits on
    one another do; a wait on a barrier is suspended by the hardware for longer than
    the products' copies take, so these calls succeed.)"""
    call, out = CASES[name]()
    call()
    assert sg.status() == sg.OK
    want = out.clone()
    try:
        for _ in range(5):
            sg.set_wait_limit(1)
            call()
            assert sg.status() in (sg.OK, sg.ERR_TIMEOUT)
            sg.set_wait_limit(0)        # the default again
            out.zero_()
            call()
            assert sg.status() == sg.OK
            assert torch.equal(out, want)
    finally:
        sg.set_wait_limit(0)


# ---- hand-overs between blocks ------------------------------------------------------

@pytest.mark.parametrize("make", [lambda: moe_case(16, 24, 4, 1096, 520), lambda: moe_case(2, 3, 3, 4096, 200),
                                  lambda: linear_case(100, 4096, 8192)])
def test_sums_of_other_blocks_are_complete_every_time(make):
    """Results that are added from several blocks' parts (experts by one warp whose lanes
    watch a column group each; parts of K by the last warp to arrive), 200 times."""
    call, out = make()
    call()
    want = out.clone()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        out.zero_()
        call()
        wrong += (out != want).sum()
    assert sg.status() == sg.OK
    assert int(wrong) == 0


# ---- rows ------------------------------------------------------------------

@pytest.mark.parametrize("K", [96, 515, 4096, 17000])
def test_norm_of_the_largest_rows_keeps_eps(K):
    """Squares that overflow FP32 are summed of scaled values; an eps of their size
    counts all the same."""
    rng = np.random.default_rng(K)
    x = (1e19 * rng.uniform(0.5, 1.5, (5, K))).astype(np.float32)
    w = np.ones(K, dtype=np.float32)
    for eps in (1e38, 3e37, 1e-6):
        run_rows(x, None, w, eps=eps, with_y=True)


@pytest.mark.parametrize("M", [2, 40])
def test_linear_without_terms_reads_no_scale(M):
    """K == 0 gives act(bias), whatever the scales hold."""
    nan = lambda n: torch.full((n,), float("nan"), device="cuda")  # noqa: E731
    b = torch.tensor([-1.0, 2.0, 0.5], device="cuda")
    out = torch.full((M, 3), 9.0, device="cuda")
    for bias, want in ((b, torch.relu(b)), (None, torch.zeros(3, device="cuda"))):
        sg.linear_q8(torch.empty((M, 0), dtype=torch.int8, device="cuda"), nan(M),
                     torch.empty((3, 0), dtype=torch.int8, device="cuda"), nan(3), out, bias=bias, activation="relu")
        assert sg.status() == sg.OK
        assert torch.equal(out, want.expand(M, 3))
