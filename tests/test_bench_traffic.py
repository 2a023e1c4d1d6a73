"""The stored counters of HBM traffic are of the present kernel sources, so that bench.py reports them."""
import importlib
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
    STORED = json.load(f)


@pytest.mark.parametrize("workload", sorted(STORED))
def test_stored_counters_are_reported(workload):
    bench = importlib.import_module("bench")
    reported = [bench.traffic_from_profiles(workload, kernel) for kernel in bench.KERNEL_SRC]
    assert STORED[workload]["hbm_bytes_per_launch"] in reported
