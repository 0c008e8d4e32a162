"""The recorded DRAM traffic belongs to the kernels that are there: bench.py reports a figure only while its kernel's sources are
those that it was taken on."""
import json
import os

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "profiles", "dram_traffic.json")) as f:
    RECORDED = json.load(f)


def test_every_kernel_of_the_benchmark_is_recorded():
    assert set(RECORDED) == set(bench.KERNEL_SOURCES)


@pytest.mark.parametrize("kernel,workload", [(k, w) for k in RECORDED for w in RECORDED[k]])
def test_recorded_traffic_is_of_the_sources_that_are_there(kernel, workload):
    entry = RECORDED[kernel][workload]
    assert entry["source_sha"] == bench.kernel_source_sha(kernel)
    assert bench.recorded_traffic(kernel, workload) == entry["dram_read"] + entry["dram_write"] > 0
