"""Which kernels bench.py may report DRAM traffic for (no GPU)."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402


def test_the_single_launch_has_no_traffic_figure():
    # ncu replays a cooperative launch without its cluster dimension: what it counts there is a
    # kernel that reads a fraction of the weights
    assert not [k for k in bench.NCU_TRAFFIC if k[1] == "k_linear_fused"]
    assert bench.ncu_traffic("dit_w4a8@T256", "k_linear_fused") is None
