"""The benchmark's DRAM traffic figure belongs to the sources it stands beside."""
import bench


def test_the_captured_traffic_is_of_these_sources():
    """A change of the listed sources needs a new capture (the command is in
    profiles/tc_gemm_pair_llama_8b_1layer.md); until then the roofline's traffic
    is null."""
    cap = bench.TRAFFIC_CAPTURES["ns_axpy"]
    assert bench.source_fingerprint(cap["sources"]) == cap["sha"]
    for workload, traffic in cap["bytes_per_pass"].items():
        assert bench.captured_traffic("ns_axpy", workload) == traffic
