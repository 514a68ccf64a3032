"""The bench's DRAM traffic comes from a profile of the attention kernel as it
stands: a change of that kernel's sources needs a new capture."""
import bench


def test_attention_profile_is_of_the_current_source():
    traffic = bench.profiled_traffic()
    assert traffic is not None, f"no profile of kernel source {bench.kernel_source_hash()}"
    assert 1e6 < traffic < 1e9
