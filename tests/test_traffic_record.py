"""The recorded DRAM traffic of the attention kernel belongs to the kernel's present sources, so that bench.py reports it."""
import bench


def test_traffic_was_taken_on_these_sources():
    rec = bench.traffic_record()
    assert rec is not None and rec["dram_bytes_per_launch"] == round(sum(rec["captured_mb"].values()) * 1e6)
