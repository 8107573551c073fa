"""The committed profile that the bench quotes belongs to the kernel sources beside it."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_the_bench_quotes_traffic_of_the_current_verify_kernel():
    import bench

    assert bench._profiled_traffic(), "the summary under profiles/ is of other kernel sources"
