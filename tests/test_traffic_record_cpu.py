"""The committed DRAM-traffic record belongs to the FP16 kernel's present sources, so the bench has its figure."""
import bench


def test_record_is_of_the_present_sources():
    traffic, note = bench.traffic_record()
    assert traffic is not None, note
    assert traffic == 1098227200 + 256536064
