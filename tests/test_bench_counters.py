"""The scans' committed counters are those of the sources here, so the bench reports them (no GPU)."""
import os

import pytest

import bench

NAMES = [f[:-5] for f in sorted(os.listdir(os.path.join(bench.ROOT, "profiles"))) if f.endswith(".json")]


def test_the_workloads_have_their_counters():
    assert {"sq_scan_long", "sq_scan_mid", "sq_scan_block", "sq_bwd_long"} <= set(NAMES)


@pytest.mark.parametrize("name", NAMES)
def test_counters_are_current(name):
    doc, note = bench.load_profile(name)
    assert doc is not None, note
    assert doc["kernels"]
