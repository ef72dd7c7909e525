"""The 8-bit feed-forward example, end to end, against the same block in FP32.

Bound on the distance.  Quantising a row rounds each value by at most half a
step of max|row|/127; over a row of normal numbers (max about 4 deviations) that
is 4 / 127 / sqrt(12) = 0.9% of its size, over a hidden row (a product of two,
max up to 10 deviations) 2.3%.  A block quantises its rows, two weights and the
hidden rows, and the gate and up products both carry the first two:
sqrt(4 * 0.9^2 + 2.3^2 + 0.9^2) = 3%.  Twice that is allowed."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import dense_fp32_matrix_row_gb300 as sg  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sg.build()
    spec = importlib.util.spec_from_file_location("q8_feed_forward", os.path.join(ROOT, "examples", "q8_feed_forward.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,hidden,inner,experts,expert_inner,top_k", [
    (1, 512, 1024, 8, 256, 2), (5, 384, 900, 5, 100, 1), (33, 256, 640, 12, 144, 4), (300, 1024, 2048, 0, 0, 0)])
def test_blocks_stay_near_fp32(example, tokens, hidden, inner, experts, expert_inner, top_k):
    result = example.run(tokens, hidden, inner, experts, expert_inner, top_k)
    assert set(result) == ({"dense", "experts"} if experts else {"dense"})
    for name, (off, _) in result.items():
        assert 0 < off < 0.06, f"{name}: {off}"
