"""The package without torch: it imports, and its host-side calls work; torch is
needed by the calls that take tensors alone."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys

class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("No module named 'torch'", name="torch")

sys.meta_path.insert(0, NoTorch())
from dense_fp32_matrix_row_gb300 import *
import dense_fp32_matrix_row_gb300 as sg
sg.build()
assert version() > 0 and select_kernel(64, 64, 64, A=1 << 30, B=2 << 30, C=3 << 30) > 0
for name in sg.__all__:
    assert callable(globals()[name]), name
for call in (lambda: quantize_q8(None, None, None), lambda: linear_q8(None, None, None, None, None)):
    try:
        call()
    except ModuleNotFoundError as e:
        assert e.name == "torch"
    else:
        raise AssertionError("a call without torch went through")
"""


def test_import_and_host_calls():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_import_leaves_torch_alone():
    """A star import loads torch no more than a plain one does."""
    program = "from dense_fp32_matrix_row_gb300 import *; import sys; assert 'torch' not in sys.modules"
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
