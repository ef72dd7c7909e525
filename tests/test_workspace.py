"""What the entry points do with their stream workspaces, on a stand-in for the
CUDA runtime (tests/c/fake_device.cpp): host threads that share a stream, and graphs."""

import os
import subprocess

import pytest


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from dense_fp32_matrix_row_gb300.build import ARCH, CSRC, NVCC_FLAGS, nvcc
    out = tmp_path_factory.mktemp("fake")
    files = [os.path.join(CSRC, f) for f in ("api.cu", "noalloc.cu", "q8_api.cu")] + [
             os.path.join(ROOT, "tests", "c", "fake_device.cpp")]
    objects = [str(out / (os.path.basename(f) + ".o")) for f in files]
    jobs = [subprocess.Popen([nvcc(), *ARCH, *NVCC_FLAGS, "-c", f, "-o", o]) for f, o in zip(files, objects)]
    assert [j.wait(300) for j in jobs] == [0] * len(jobs)
    exe = str(out / "fake_device")
    subprocess.run([nvcc(), "-cudart", "none", *objects, "-o", exe, "-Xlinker", "-lpthread"], check=True, timeout=300)
    return exe


def run(program, scenario):
    r = subprocess.run([program, scenario], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("scenario", ["threads_share_a_stream", "threads_on_their_own_streams",
                                      "per_thread_streams_share_nothing"])
def test_host_threads(program, scenario):
    run(program, scenario)


@pytest.mark.parametrize("scenario", ["graph_keeps_its_workspace", "growth_frees_the_old_workspace"])
def test_capture(program, scenario):
    run(program, scenario)
