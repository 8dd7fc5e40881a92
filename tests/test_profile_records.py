"""The committed traffic records describe the current kernels: bench.py prints a record only
while the hash of its kernel sources matches, so one that no longer does is lost without a
word.  A change to those sources takes its records again."""
import glob
import json
import os

import pytest

import bench

RECORDS = sorted(glob.glob(os.path.join(bench.PROFILES, "traffic_*.json")))


def test_there_are_records():
    assert len(RECORDS) >= 8


@pytest.mark.parametrize("path", RECORDS, ids=os.path.basename)
def test_record_is_of_the_current_sources(path):
    rec = json.load(open(path))
    name = os.path.basename(path)[len("traffic_"):-len(".json")]
    stage = "gate_up"
    assert name == f"{stage}_{rec['workload']}"
    assert bench.measured_traffic(rec["workload"], stage) == rec["bytes_per_launch"] > 0
