"""The recorded DRAM traffic belongs to the kernels as they are: bench.py leaves it
out of its line once the code that a kernel is compiled from has changed."""

import json
import os

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORD = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))
ENTRIES = [(kernel, workload) for kernel, w in RECORD.items() if not kernel.startswith("_") for workload in w]


@pytest.mark.parametrize("kernel,workload", ENTRIES)
def test_record_is_of_the_current_source(kernel, workload):
    assert bench.ncu_traffic(kernel, workload) == RECORD[kernel][workload]["dram_bytes_per_launch"]
