"""The HBM traffic records that the benchmark reports belong to the present
kernels: each is kept with the hash of its kernel's sources."""
import json
import os

import pytest

import bench
from layer_lstm_amd import profile_summary

RECORDS = json.load(open(bench.TRAFFIC_FILE))


@pytest.mark.parametrize("workload", sorted(RECORDS))
def test_records_are_of_the_present_sources(workload):
    assert set(RECORDS[workload]) <= set(profile_summary.KINDS) and os.path.exists(bench.TRAFFIC_FILE)
    for kind, rec in RECORDS[workload].items():
        assert bench.traffic_for(workload, kind) == rec["bytes_per_launch"] > 0, kind
