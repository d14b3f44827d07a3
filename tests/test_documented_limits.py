"""The size limits that include/ssm.h states for linear attention and layer norm: just inside, only a missing pointer is
refused; just outside, the size is (no GPU; nothing is enqueued)."""
import os

import pytest

import selective_state_space_35_amd as ssm
from tests.test_linattn_host import DIM, FAKE, NULL, bwd, fwd, norm, norm_bwd, update

pytestmark = pytest.mark.skipif(not os.path.exists(ssm.library_path()), reason="libssm.so not built")
ONE = dict(b=1, H=1, G=1, Dk=1, Dv=1)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_sequences(call):
    lib = ssm.load_library()
    for inside, outside in ((dict(ONE, L=2 ** 31 - 4097), dict(ONE, L=2 ** 31 - 4096)),
                            (dict(ONE, H=65535, L=8), dict(ONE, H=65536, L=8)),
                            (dict(ONE, b=2 ** 21, L=8), dict(ONE, b=2 ** 21 + 1, L=8)),
                            # b (L / 256 + 1) (H / 16 + 1) = 2^24 - 1 and 2^24
                            (dict(ONE, b=2 ** 12 - 1, L=256 * 2 ** 12), dict(ONE, b=2 ** 12, L=256 * (2 ** 12 - 1)))):
        assert call(lib, **dict(inside, q=None)) == NULL, inside
        assert call(lib, **dict(outside, q=None)) == DIM, outside


def test_tokens_and_norms():
    lib = ssm.load_library()
    assert update(lib, b=2 ** 21, H=1, G=1, state=None) == NULL and update(lib, b=2 ** 21 + 1, H=1, G=1, state=None) == DIM
    for call in (norm, norm_bwd):
        for inside, outside in ((dict(rows=2 ** 31 - 1), dict(rows=2 ** 31)), (dict(rows=2 ** 21, H=2 ** 9), dict(rows=2 ** 21, H=2 ** 10)),
                                (dict(W=16384), dict(W=16385)), (dict(H=2 ** 21, W=511), dict(H=2 ** 21, W=512)),
                                (dict(H=2 ** 16, W=2 ** 14 - 1), dict(H=2 ** 16, W=2 ** 14))):
            assert call(lib, **dict(inside, x=None)) == NULL, inside
            assert call(lib, **dict(outside, x=None)) == DIM, outside
    assert FAKE % 256 == 0
