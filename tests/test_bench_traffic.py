"""The benchmark reports a kernel's measured DRAM bytes only while its sources are those that were measured:
a change elsewhere must not drop them."""
import pytest

import bench


@pytest.mark.parametrize("workload,stage", [("csa_decode", "index_topk"), ("csa_decode", "attn"), ("hca_prefill", "attn")])
def test_measured_traffic_belongs_to_the_sources(workload, stage):
    assert bench.kernel_traffic(workload, stage, "auto") > 0
