"""The DRAM bytes that bench.py reports were captured on the kernels that are here: an entry whose kernel, or
a header that all kernels share, has changed since is captured again or taken out."""
import json

import pytest

import bench

with open(bench.TRAFFIC_FILE) as f:
    ENTRIES = sorted(json.load(f))


@pytest.mark.parametrize("entry", ENTRIES)
def test_traffic_is_of_the_present_kernels(entry):
    kernel, workload = entry.split("@")
    assert bench.traffic_for(kernel, workload)
