"""The counted traffic that bench.py reports beside its times."""
import glob
import os
import re

import pytest

import bench

SUMMARIES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(bench.PROFILES, "moe_layer_*_counters.txt")))


@pytest.mark.parametrize("stage", sorted(bench.STAGE_SOURCES))
@pytest.mark.parametrize("name", SUMMARIES)
def test_committed_counters_are_of_the_current_kernels(name, stage):
    """A summary whose kernel sources have changed since it was taken is left out of the line: then take it anew."""
    text = open(os.path.join(bench.PROFILES, name)).read()
    if not re.search(rf"^{stage}_hbm_bytes_per_launch:", text, re.M):
        pytest.skip("this workload has no such launch")
    assert bench.read_traffic(re.fullmatch(r"moe_layer_(.*)_counters\.txt", name)[1], stage) > 0
