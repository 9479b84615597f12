"""The benchmark's measured DRAM traffic belongs to the sources of the layer's GEMM that it was captured with."""
import sys

from helpers import ROOT

sys.path.insert(0, ROOT)


def test_the_default_workloads_traffic_is_that_of_the_sources():
    import bench
    name = "dsv4_flash_decode_T64"
    assert bench.W1_TRAFFIC[name][1] == bench.gemm_sources_sha(), "the GEMM's sources changed: capture its traffic again"
    assert bench.w1_traffic(name) == bench.W1_TRAFFIC[name][0]
