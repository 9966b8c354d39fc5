"""The captured DRAM traffic that bench.py reports belongs to the kernels' sources as they are: a capture whose
sources have changed since is not reported, and has to be taken again."""
import os

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "profiles", "traffic.txt")) as f:
    WORKLOADS = [line.split()[0].split("=", 1)[1] for line in f if line.startswith("workload=")]


def test_the_default_line_has_a_capture():
    assert "moe" in WORKLOADS


@pytest.mark.parametrize("workload", WORKLOADS)
def test_capture_is_of_these_sources(workload):
    got, fields = bench.kernel_traffic(workload)
    assert got is not None and got > 0 and fields["workload"] == workload
