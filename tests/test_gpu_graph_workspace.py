"""A captured call's workspace outlives later calls that need a larger one."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.build()


def int8(*shape):
    return torch.randint(-90, 91, shape, device="cuda", dtype=torch.int8)


def test_replay_after_the_stream_workspace_grew():
    torch.manual_seed(5)
    stream = torch.cuda.Stream()
    T, H, inner, N = 8, 256, 192, 8192
    x, router = torch.randn((T, H), device="cuda"), torch.randn((6, H), device="cuda")
    w_up, w_down = int8(6, 2 * inner, H), int8(6, H, inner)
    s_up, s_down = torch.full((6, 2 * inner), 1e-3, device="cuda"), torch.full((6, H), 1e-3, device="cuda")
    xq, wq = int8(9000, 1024), int8(N, 1024)
    xs, ws = torch.ones(9000, device="cuda"), torch.ones(N, device="cuda")
    out, big = torch.zeros((T, H), device="cuda"), torch.empty((9000, N), device="cuda")

    def experts():
        sg.moe_q8(x, router, w_up, s_up, w_down, s_down, out, 2, stream=stream)

    def prompt(rows):
        sg.linear_q8(xq[:rows], xs[:rows], wq, ws, big[:rows], stream=stream)

    torch.cuda.synchronize()
    graphs, want = [], None
    for rows in (200, 3000, 9000):      # the last two need larger workspaces than the graphs before them have
        prompt(rows)
        experts()
        assert sg.status(stream) == sg.OK
        want = out.clone() if want is None else want
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            experts()
        graphs.append(graph)
        for g in graphs:
            with torch.cuda.stream(stream):
                out.zero_()
                prompt(rows)
                g.replay()
                prompt(rows)
            assert sg.status(stream) == sg.OK
            assert torch.equal(out, want)
    del graphs, g, graph
    torch.cuda.synchronize()
    assert sg.release_workspaces() == sg.OK
