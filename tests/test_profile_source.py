"""The profiled traffic of the expert GEMM belongs to the kernel source in the tree:
otherwise the bench reports none."""
import os

import bench


def test_profiled_traffic_is_of_this_source():
    assert bench.ffn_source_sha16() == bench.FFN_TRAFFIC["kernel_sha16"]
    with open(os.path.join(bench.ROOT, bench.FFN_TRAFFIC["profile"])) as f:
        assert bench.FFN_TRAFFIC["kernel_sha16"] in f.read()
