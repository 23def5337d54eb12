"""The recorded DRAM traffic of the expert GEMMs belongs to the kernels as they are: bench.py
reports it only while their sources hash as they did."""

import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

with open(bench.PROFILE_TRAFFIC) as fh:
    RECORDS = [(w, k) for w, kernels in json.load(fh).items() if not w.startswith("_") for k in kernels]


@pytest.mark.parametrize("workload,kernel", RECORDS)
def test_recorded_traffic_is_reported(workload, kernel):
    assert bench.profiled_traffic(workload, kernel) > 0
