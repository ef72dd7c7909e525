"""The 8-bit operators at the ends of their ranges."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402


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
