"""The committed traffic counters of the w13 GEMM are those of its present
sources, so that bench.py reports them (no GPU).  Whoever changes one of those
sources takes the counters anew; what other kernels share has headers of its
own."""
import os
import sys

import moe_inputs as mi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_traffic_of_the_present_sources_is_reported():
    got = bench.measured_traffic()
    assert got is not None
    assert got["total"] == got["read"] + got["write"] >= bench.w13_algorithmic_bytes(mi.spec("denoise_1micro"))
