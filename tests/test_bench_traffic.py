"""The DRAM traffic that the bench reports beside a kernel's roofline belongs to the sources that the kernel is built
from: a change of a header that the kernel's record is dated by takes its figure out of every line of the bench."""
import json
import os

import bench


def test_recorded_traffic_is_of_the_current_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        records = json.load(f)
    assert records
    for key, record in records.items():
        kernel, workload = key.split(":", 1)
        assert bench.recorded_traffic(kernel, workload) == record["dram_bytes_per_launch"], key
