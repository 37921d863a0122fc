"""The benchmark's measured traffic holds for the sources that are here: every
kernel of the default workload has its record, stamped with their digest."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


def test_the_default_workload_has_its_traffic():
    kernels = [k.split("@")[0] for k in json.load(open(bench.TRAFFIC_FILE)) if k.endswith("@moe-experts-bf16")]
    assert "rans_decode" in kernels and "rans_encode" in kernels
    for k in kernels:
        assert bench.measured_traffic(k, "moe-experts-bf16"), k


def test_the_version_is_no_part_of_the_digest():
    """It is the header's: a new one changes no kernel."""
    root = os.path.dirname(bench.TRAFFIC_FILE)
    lib = open(os.path.join(os.path.dirname(root), "lossless_weight_compression_bf16_amd", "csrc", "wc_lib.hip")).read()
    assert "return WC_VERSION;" in lib and "kVersion" not in lib
