"""The committed DRAM counters of the GEMV sweep belong to the GEMV sources as
they are: bench.py reports them only while the code of those files has not
changed since they were taken."""
import bench


def test_committed_traffic_matches_the_sources():
    assert bench.committed_traffic() is not None, (
        "code of " + ", ".join(bench.GEMV_SOURCES) + " changed: profiles/q4k_gemv_sweep_traffic.json has to be taken again "
        "(what other kernels need belongs into headers of their own)")
