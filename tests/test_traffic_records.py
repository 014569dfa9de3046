"""The benchmark reports a kernel's measured DRAM bytes only where the record
in profiles/ was taken on the current sources (the kernel's file and the two
headers that it includes).  A change there has to bring the record along: taken
again, or with its hash brought up to date where the device code is the same."""
from __future__ import annotations

import glob
import json
import os

import pytest

import bench

RECORDS = sorted(glob.glob(os.path.join(bench.ROOT, "profiles",
                                        "*_traffic.json")))


@pytest.mark.parametrize("path", RECORDS, ids=os.path.basename)
def test_record_is_of_the_current_sources(path):
    with open(path) as fh:
        record = json.load(fh)
    assert record["entries"]
    for e in record["entries"]:
        assert bench.read_traffic(record["kernel"], e["bench_workload"]) == \
            e["dram_bytes_per_launch"]
