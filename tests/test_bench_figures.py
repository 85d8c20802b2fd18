"""bench.py's stored memory traffic was measured with the kernel sources as they are."""


def test_traffic_figures_are_of_the_current_sources():
    import bench
    assert bench._kernel_sources_sha() == bench.TRAFFIC["sources_sha"]
