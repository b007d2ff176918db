"""Host-side check that bench.py has a traffic figure to report: profiles/traffic.json was taken with the kernels' present sources
(profiles/k_gemv_k_gemm_attn4096_traffic.md has the two counter runs that write it)."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("key", sorted(bench.TRAFFIC_KERNELS))
def test_counters_are_of_the_present_sources(key):
    assert bench.traffic_from_profile(key) is not None
