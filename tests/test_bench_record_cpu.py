"""The benchmark's committed records belong to the sources they were taken on (no GPU needed)."""
import bench


def test_traffic_record_is_of_the_current_gemm():
    """The roofline's DRAM traffic is reported only for the GEMM sources it was captured on; after a
    change there it is captured again (profiles/expert_gemms_skewed_e64_top6_t4096.md has the
    commands)."""
    for kernel in ("expert_gemm1", "expert_gemm2"):
        assert bench.traffic_record(kernel, "skewed_e64_top6"), kernel
    assert bench.traffic_record("expert_gemm1", "another workload") is None
