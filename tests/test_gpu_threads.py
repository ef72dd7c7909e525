"""Entry points called from several host threads at once, on one stream and on the
stream that each thread has of its own."""

import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


def int8(gen, *shape):
    return torch.randint(-90, 91, shape, generator=gen, device="cuda", dtype=torch.int8)


def calls(seed, stream):
    """An expert layer, a product on the tiles and an FP32 product, of sizes and
    values of this seed: ([call], their outputs)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    T, H, inner, M, N = 4 + seed, 256, 192, 40 + 16 * seed, 4500
    x, router = normal(T, H), normal(6, H)
    w_up, w_down = int8(gen, 6, 2 * inner, H), int8(gen, 6, H, inner)
    s_up, s_down = torch.full((6, 2 * inner), 1e-3, device="cuda"), torch.full((6, H), 1e-3, device="cuda")
    xq, wq = int8(gen, M, H), int8(gen, N, H)
    xs, ws = torch.ones(M, device="cuda"), torch.full((N,), 1e-3, device="cuda")
    a, b = normal(M, H), normal(H, 512)
    out = [torch.zeros((T, H), device="cuda"), torch.zeros((M, N), device="cuda"), torch.zeros((M, 512), device="cuda")]
    return [lambda: sg.moe_q8(x, router, w_up, s_up, w_down, s_down, out[0], 2, stream=stream),
            lambda: sg.linear_q8(xq, xs, wq, ws, out[1], stream=stream),
            lambda: sg.sgemm(a, b, out[2], stream=stream)], out


PER_THREAD = 2      # the handle cudaStreamPerThread


@pytest.mark.parametrize("stream", ["shared", PER_THREAD])
def test_threads_get_their_own_results(stream):
    if stream == "shared":
        stream = torch.cuda.Stream()
    work = [calls(seed, stream) for seed in range(4)]
    torch.cuda.synchronize()
    for todo, _ in work:
        for call in todo:
            call()
    assert sg.status(stream) == sg.OK
    want = [[t.clone() for t in out] for _, out in work]
    for _, out in work:
        for t in out:
            t.zero_()
    sg.release_workspaces()          # the threads grow the workspace as well
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(work))

    def thread(todo):
        try:
            start.wait()
            for _ in range(50):
                for call in todo:
                    call()
            assert sg.status(stream) == sg.OK
        except Exception as e:      # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(todo,)) for todo, _ in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for (_, out), w in zip(work, want):
        assert all(torch.equal(g, h) for g, h in zip(out, w))
    assert sg.release_workspaces() == sg.OK
