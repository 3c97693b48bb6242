"""The bench reports the forward's DRAM traffic from a recorded profile as long as the record is of the present source."""
import bench


def test_the_default_workload_has_its_traffic_record():
    assert bench.recorded_traffic("sa_forward_kernel", "sweep69k_top20")
