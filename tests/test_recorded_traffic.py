"""The DRAM traffic that the bench reports is recorded for the grouped GEMMs of this tree (CPU only)."""
import json
import os

import bench


def test_recorded_traffic_is_that_of_the_present_kernels():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        rec = json.load(f)
    assert rec["kernel_source_hash"] == bench.kernel_source_hash()
    for workload, stages in rec["per_launch_bytes"].items():
        for stage, nbytes in stages.items():
            assert bench.recorded_traffic(workload, stage) == nbytes
