"""The example's attention block on the GPU: prompt and decode step, over head
layouts, stay near the same block in FP32."""

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
    spec = importlib.util.spec_from_file_location("q8_attention", os.path.join(ROOT, "examples", "q8_attention.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("sequences,context,hidden,heads,kv_heads,dim", [(3, 70, 512, 8, 2, 64), (1, 300, 1024, 4, 4, 128),
                                                                        (2, 33, 640, 10, 1, 80)])
def test_distance_from_fp32(example, sequences, context, hidden, heads, kv_heads, dim):
    """Quantising a row of normal numbers rounds it by 0.9% of its size (half a step of
    1/127 of about 4 deviations, spread evenly: 4 / 127 / sqrt(12)).  Queries, keys
    and values carry the token's and the weights' rounding (1.3%), keys and values
    their own (1.6%).  A score is the product of a query and a key, 2.1% off in a size of
    1.5^2 (both norms' weights), so 4.7%, and each probability by as much; independent
    from token to token, that is what the weighted sum is off by.  With the values'
    1.6% and the last product's rows and weights (1.3%): 5.1%.  Twice that is allowed."""
    for name, (off, us) in example.run(sequences, context, hidden, heads, kv_heads, dim).items():
        assert 0 < off < 0.1, (name, off)
        assert us is None
    assert sg.status() == sg.OK


def test_replayed_step(example):
    result = example.run(4, 100, 512, 8, 2, 64, repeats=3)
    assert result["decode"][1] > 0
