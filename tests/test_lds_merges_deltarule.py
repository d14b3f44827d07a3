"""The guard of tests/test_lds_merges.py against a miscompile of paired LDS accesses, over the sources of the gated delta rule
and of the norms around a block (CPU only: compiles, runs nothing)."""
import os
import shutil

import pytest

from tests import test_lds_merges as guard


@pytest.mark.timeout(900)
@pytest.mark.skipif(not shutil.which(guard.HIPCC) and not os.path.exists(guard.HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("source,least", [("ssm_deltarule.hip", 1000), ("ssm_blocknorm.hip", 1)])
def test_merged_lds_accesses_keep_their_offsets(source, least):
    merged, problems = guard._check(source)
    assert not problems, "\n".join(problems[:20])
    assert merged >= least  # the check is not vacuous
