"""bench.py's recorded DRAM traffic is of the kernel sources in the tree: its
JSON line leaves the figure out where a source has changed since the capture."""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.NCU_TRAFFIC))
def test_recorded_traffic_is_reported(kernel):
    assert bench.captured_traffic(kernel, "config3") == bench.NCU_TRAFFIC[kernel]["bytes"]
