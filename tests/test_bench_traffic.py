"""The DRAM bytes that bench.py reports were captured from the image attention's kernels as they are (CPU)."""
import bench


def test_traffic_belongs_to_the_kernels_as_they_are():
    """Sources and headers of other operators leave the recorded bytes valid."""
    for key, (src, sha, nbytes) in bench.TRAFFIC.items():
        assert bench.measured_traffic(key) == nbytes, f"{src} or a header of it changed: capture its traffic again"
