"""The DRAM traffic that bench.py reports belongs to the decode kernel that is
there: each summary is keyed by a hash of the kernel's source."""
import glob
import json
import os

import pytest

import bench

SUMMARIES = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "*_traffic.json")))


@pytest.mark.parametrize("path", SUMMARIES, ids=os.path.basename)
def test_traffic_summaries_were_taken_on_the_current_source(path):
    d = json.load(open(path))
    assert d["kernel_source_hash"] == bench.kernel_source_hash()
    assert bench.profiled_traffic(d["workload"], d["kernel"]) == d["dram_bytes_per_launch"] > 0


def test_the_default_workload_has_a_summary():
    assert bench.profiled_traffic("short") is not None
