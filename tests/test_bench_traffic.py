"""The traffic figures that bench.py reports belong to the kernel sources they
were taken on: work elsewhere leaves those sources as they are."""
import bench


def test_traffic_figures_belong_to_these_sources():
    name = "gptoss_b2_h16_d64_w128_s8192"
    assert bench.measured_traffic(name) == bench.MAIN_TRAFFIC[name]["bytes"]
    assert bench.measured_traffic(name, bench.FWD_TRAFFIC, bench.FWD_SOURCES) == bench.FWD_TRAFFIC[name]["bytes"]
