"""The committed profiles stand for the kernels as they are."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


@pytest.mark.parametrize("workload", ["llama8b_step", "llama8b_step_fp8", "skewed", "token_sparse"])
def test_traffic_of_the_decode_kernel_is_of_its_present_sources(workload):
    """bench.py reports a profile's DRAM bytes only while the decode kernel's sources are those it was
    taken on: what other kernels need goes to files of their own."""
    assert bench.traffic_from_profile(workload) > 0
