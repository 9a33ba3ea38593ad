"""The counter summary that bench.py reports HBM traffic from is the one of the kernel sources that are
there: after a change to one of them the counters are taken again (bench.py --traffic-run under the
profiler), or the benchmark's line says null."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("cls", sorted(bench.C5_KERNEL))
def test_traffic_is_reported(cls):
    assert bench.gemm_traffic(cls) is not None
