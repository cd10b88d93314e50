"""The DRAM traffic that bench.py reports comes from committed captures, each valid for the sources it names: a change to one
of them silences the figure until it is taken again (no GPU needed)."""

import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_traffic_record_is_of_the_present_sources():
    records = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))
    assert records
    for kernel, r in records.items():
        assert os.path.exists(os.path.join(ROOT, r["capture"])), kernel
        assert bench.ncu_traffic(kernel) == r["bytes_per_launch_full"], f"{kernel}: sources changed since its capture"
