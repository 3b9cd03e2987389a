"""The recorded traffic of the profiled kernels (CPU)."""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402


def test_recorded_traffic_is_that_of_the_current_sources():
    """The bench gives the traffic that was measured on these very kernels; a change of a shared header that they
    do not need would take it away."""
    for kernel, name in (("decode_step", "qwen3_14b_gate"), ("decode_step", "r1_7b_256k"), ("decode_step", "qwen3_4b"),
                         ("decode_step", "paged_b8"), ("rectify", "r1_7b_256k")):
        assert bench.recorded_traffic(kernel, name) is not None, (kernel, name)
