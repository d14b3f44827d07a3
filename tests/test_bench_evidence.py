"""The scans' committed counters are dropped when the scans' sources change, and only then (no GPU)."""
import os
import shutil

import pytest

import bench


@pytest.fixture
def tree(tmp_path, monkeypatch):
    src = os.path.join(bench.ROOT, "selective_state_space_35_amd", "csrc")
    dst = tmp_path / "selective_state_space_35_amd" / "csrc"
    shutil.copytree(src, dst)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return dst


@pytest.mark.parametrize("name,counts", [("ssm_kernels.hip", True), ("ssm_fused.hip", True), ("ssm_bwd.hip", True), ("ssm_chain.h", True),
                                         ("ssm_device.h", True), ("ssm_internal.h", True), ("ssm_api.hip", False),
                                         ("ssm_linattn.hip", False), ("ssm_layernorm.hip", False)])
def test_a_change_of(name, counts, tree):
    before = bench.source_hash()
    with open(tree / name, "a") as f:
        f.write("// another line\n")
    assert (bench.source_hash() != before) == counts


def test_the_scans_share_nothing_with_what_does_not_count(tree):
    """No counted source includes one that does not count."""
    for f in os.listdir(tree):
        if f not in bench.HASH_EXCLUDES:
            text = open(tree / f).read()
            for e in bench.HASH_EXCLUDES:
                assert f'#include "{e}"' not in text, (f, e)
