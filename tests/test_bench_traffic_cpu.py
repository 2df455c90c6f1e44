"""The combine's captured DRAM bytes that the benchmark reports belong to the
kernel as it is: a change of its sources drops them, and a helper that only
other kernels use does not belong in those files."""
import bench


def test_the_captured_traffic_stands():
    t = bench.COMBINE_TRAFFIC
    assert bench.combine_traffic(t["algorithmic_bytes"]) == t["bytes"]
