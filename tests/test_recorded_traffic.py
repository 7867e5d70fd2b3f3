"""The DRAM traffic recorded for the benchmark's kernels holds for the sources they are built from: a change of those
sources has to bring a new record, or the benchmark's line loses the figure."""
import json
import os

import bench


def test_every_record_is_of_the_current_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        records = json.load(f)
    assert set(records) == set(bench.KERNEL_SOURCES)
    for kernel, record in records.items():
        assert bench.recorded_traffic(kernel) == record["dram_bytes_per_launch"], kernel
