"""The bench's record of measured DRAM traffic belongs to the kernel sources of the tree: where one
of them changed since the capture, the bench has no traffic figure."""
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bench  # noqa: E402


def test_the_traffic_record_is_of_these_sources():
    traffic = bench.measured_traffic()
    assert traffic is not None, "re-capture the wave kernel's DRAM bytes (see bench.py)"
    # within a tenth of the bytes that the wave must move (part of its writes stays in L2)
    must = bench.algorithmic_bytes(32768, 16, 32, 128, 32, 32)
    assert 0.9 * must <= traffic <= 1.1 * must
