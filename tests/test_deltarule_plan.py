"""The tests' account of how the gated delta rule deals a call out, against the library's workspace query (no GPU)."""
import os
import random

import pytest

import selective_state_space_35_amd as ssm
from tests import deltarule_plan as plan


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspace_is_as_planned(dtype):
    if not os.path.exists(ssm.library_path()):
        pytest.skip("libssm.so not built")
    rng = random.Random(7)
    kinds = set()
    for _ in range(400):
        G = rng.randint(1, 9)
        H = G * rng.choice([1, 2, 3, 4, 6])
        b, L = rng.randint(1, 40), rng.choice([0, 1, 64, rng.randint(1, 300), rng.randint(1, 9000)])
        Dk, Dv = rng.randint(1, 128), rng.randint(1, 128)
        kinds.add((plan.cut(b, L, H, Dk, Dv, dtype)[0] > 1, 1 if H == G else min(2, plan.heads_together(b, L, H, G, dtype))))
        for backward in (False, True):
            got = ssm.ssm_deltarule_workspace(b, L, H, G, Dk, Dv, dtype, backward)
            assert got == plan.workspace(b, L, H, G, Dk, Dv, dtype, backward), (b, L, H, G, Dk, Dv, dtype, backward)
    assert len(kinds) >= 3
