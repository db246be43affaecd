"""The bench reports DRAM traffic for every kernel in its table: the committed capture is of the sources as they are.

A change to a kernel's sources voids its entry (the bench then reports none), so the capture belongs to the
change: the commands stand in profiles/dram_traffic_bench_kernels.md.
"""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_capture_is_of_these_sources(kernel):
    assert bench.kernel_traffic(kernel), f"{kernel}: its sources changed since profiles/ncu_traffic.json was captured"
