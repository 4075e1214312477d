"""The traffic that bench.py reports beside its roofline was counted on the GEMM's present sources: with others it reports none."""
import json

import bench


def test_counted_traffic_is_of_these_sources():
    with open(bench.TRAFFIC_FILE) as f:
        assert json.load(f)["kernel_hash"] == bench.kernel_hash()
