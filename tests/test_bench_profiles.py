"""The benchmark's committed counter summaries belong to the table's kernels as they are."""
import glob
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_counter_summaries_match_the_kernel_sources():
    sys.path.insert(0, ROOT)
    import bench
    sums = glob.glob(os.path.join(ROOT, "profiles", "*_counters.txt"))
    assert sums
    for path in sums:
        lines = open(path).read().splitlines()
        assert f"source_hash={bench.kernel_source_hash()}" in lines, path
