"""The HBM bytes per launch that bench.py reports for the step's GEMMs: those of the
committed counter summary, each at least what its operands and output take."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402
from fp8_mixed_precision_linear_amd import datagen  # noqa: E402


@pytest.mark.parametrize("cls", ["delayed fwd", "delayed dgrad", "delayed wgrad", "block fwd", "block dgrad", "block wgrad"])
def test_traffic_is_per_launch(cls, monkeypatch):
    with open(bench.TRAFFIC_JSON) as f:
        t = json.load(f)
    # (whatever state the kernel sources are in)
    monkeypatch.setattr(bench, "traffic_sources_sha256", lambda: t["sources_sha256"])
    least, T = 0.0, 8192
    for di, do in (datagen.C5_LINEARS[n] for n in bench.C5_ORDER):
        out = {"fwd": 2 * T * do, "dgrad": 2 * T * di, "wgrad": 4 * di * do}[cls.split()[1]]
        operands = {"fwd": T * di + di * do, "dgrad": T * do + di * do, "wgrad": T * di + T * do}[cls.split()[1]]
        least += (operands + out) / 5
    got = bench.gemm_traffic(cls)
    assert got == t["kernels"][cls]["traffic_bytes"] and got >= least
    assert t["kernels"][cls]["algorithmic_bytes"] == round(least)


def test_traffic_of_other_sources_is_not_reported(monkeypatch):
    monkeypatch.setattr(bench, "traffic_sources_sha256", lambda: "0" * 64)
    assert bench.gemm_traffic("block wgrad") is None
