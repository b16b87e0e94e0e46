"""CPU test: the benchmark's DRAM traffic records belong to the sources as they
are (an edit that changes a kernel's code wants a new capture, any other a new
source_sha; otherwise the benchmark reports null)."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


@pytest.mark.parametrize("kernel", sorted(bench.NCU_TRAFFIC))
def test_records_are_current(kernel):
    e = bench.NCU_TRAFFIC[kernel]
    assert e["source_sha"] == bench.kernel_source_sha(e["sources"])
