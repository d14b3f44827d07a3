"""Host-side checks of the gated delta rule's entry points: no GPU needed.

Refusals come back as the documented ssm_status before anything is enqueued, sizes that are nothing to do return without
looking at pointers, the workspace query refuses what the calls refuse, the documented size limits are where the header says,
and the binding names the argument that does not fit.
"""
import os

import pytest

import selective_state_space_35_amd as ssm

OK, NULL, DIM, DTYPE, ALIGN, SCRATCH = 0, -1, -2, -3, -5, -8
FAKE = 0x10000  # never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.library_path()):
        pytest.skip("libssm.so not built")
    return ssm.load_library()


def fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, beta=None, g=None, A=None, lengths=None, scale=1.0, h0=None, y=FAKE, last=None, b=1, L=8,
             H=4, G=2, Dk=64, Dv=64, dtype=1, ws=None, n=0, stream=None)
    a.update(kw)
    return lib.ssm_deltarule_fwd(*a.values())


def bwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, beta=None, g=None, A=None, lengths=None, scale=1.0, h0=None, dy=FAKE, dlast=None, dq=FAKE,
             dk=FAKE, dv=FAKE, dbeta=None, dg=None, dh0=None, b=1, L=8, H=4, G=2, Dk=64, Dv=64, dtype=1, ws=None, n=0, stream=None)
    a.update(kw)
    return lib.ssm_deltarule_bwd(*a.values())


def update(lib, **kw):
    a = dict(state=FAKE, q=FAKE, k=FAKE, v=FAKE, beta=None, g=None, A=None, lengths=None, scale=1.0, y=FAKE, b=1, H=4, G=2,
             Dk=64, Dv=64, dtype=1, stream=None)
    a.update(kw)
    return lib.ssm_deltarule_update(*a.values())


SIZES = [dict(b=-1), dict(H=-1), dict(G=0), dict(G=3), dict(G=-2), dict(Dk=0), dict(Dk=129), dict(Dv=0), dict(Dv=129),
         dict(H=65536, G=1), dict(b=1 << 40), dict(b=1 << 49)]


@pytest.mark.parametrize("call", [fwd, bwd, update])
def test_refusals(lib, call):
    for s in SIZES:
        assert call(lib, **s) == DIM, s
    assert call(lib, dtype=2) == DTYPE and call(lib, dtype=-1) == DTYPE
    names = {fwd: ("q", "k", "v", "y"), bwd: ("q", "k", "v", "dy", "dq", "dk", "dv"),
             update: ("state", "q", "k", "v", "y")}[call]
    for n in names:
        assert call(lib, **{n: None}) == NULL, n
    for n in ("q", "k", "v", "g", "beta"):
        assert call(lib, **{n: FAKE + 1}) == ALIGN, n
        assert call(lib, **{n: FAKE + 2, "dtype": 0}) == ALIGN, n
    for n in ("A", "lengths", "h0" if call is not update else "state"):
        assert call(lib, **{n: FAKE + 2}) == ALIGN, n
    nothing = dict.fromkeys(names)
    assert call(lib, b=0, **nothing) == OK
    assert call(lib, H=0, G=0, **nothing) == OK


@pytest.mark.parametrize("call", [fwd, bwd])
def test_sequence_refusals(lib, call):
    assert call(lib, L=-1) == DIM
    assert call(lib, L=1 << 45) == DIM
    assert call(lib, b=1 << 20, L=1 << 30) == DIM
    assert call(lib, ws=FAKE, n=-1) == SCRATCH and call(lib, ws=FAKE, n=16) == SCRATCH
    need = ssm.ssm_deltarule_workspace(1, 8, 4, 2, 64, 64, "bf16", call is bwd)
    assert need > 16 and call(lib, ws=FAKE + 128, n=need) == ALIGN and call(lib, ws=FAKE, n=need - 1) == SCRATCH


def test_backward_outputs(lib):
    for n in ("dq", "dk", "dv", "dy"):
        assert bwd(lib, **{n: FAKE + 1}) == ALIGN, n
    assert bwd(lib, dg=FAKE + 1, g=FAKE) == ALIGN and bwd(lib, dbeta=FAKE + 1, beta=FAKE) == ALIGN
    assert bwd(lib, dh0=FAKE + 2) == ALIGN and bwd(lib, dlast=FAKE + 1) == ALIGN


def test_workspace(lib):
    for s in SIZES + [dict(L=-1)]:
        a = dict(b=1, L=8, H=4, G=2, Dk=64, Dv=64)
        a.update(s)
        with pytest.raises(ssm.SSMError):
            ssm.ssm_deltarule_workspace(**a)
    with pytest.raises(ssm.SSMError):
        ssm.ssm_deltarule_workspace(1, 8, 4, 2, 64, 64, dtype=5)
    assert ssm.ssm_deltarule_workspace(0, 8, 4, 2, 64, 64) == 0
    small, large = (ssm.ssm_deltarule_workspace(1, n, 4, 2, 64, 64, backward=True) for n in (100, 100000))
    assert 0 < small < large


@pytest.mark.parametrize("call", [fwd, bwd])
def test_documented_limits(lib, call):
    """Just inside, only a missing pointer is refused; just outside, the size is."""
    one = dict(b=1, H=1, G=1, Dk=1, Dv=1)
    for inside, outside in ((dict(one, H=65535, L=8), dict(one, H=65536, L=8)),
                            (dict(one, b=2 ** 21, L=8), dict(one, b=2 ** 21 + 1, L=8)),
                            # b H (L / C + 1) = 2^23 - 1 and 2^23
                            (dict(one, L=64 * (2 ** 23 - 1) - 1), dict(one, L=64 * (2 ** 23 - 1))),
                            (dict(one, L=32 * (2 ** 23 - 1) - 1, dtype=0), dict(one, L=32 * (2 ** 23 - 1), dtype=0)),
                            (dict(one, b=2 ** 12, H=2 ** 9, G=1, L=191), dict(one, b=2 ** 12, H=2 ** 9, G=1, L=192))):
        assert call(lib, **dict(inside, q=None)) == NULL, inside
        assert call(lib, **dict(outside, q=None)) == DIM, outside
    assert update(lib, b=2 ** 21, H=1, G=1, state=None) == NULL and update(lib, b=2 ** 21 + 1, H=1, G=1, state=None) == DIM


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    if not os.path.exists(ssm.library_path()):
        pytest.skip("libssm.so not built")
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_deltarule_fwd(z(1, 4, 2, 8), z(1, 4, 2, 8), z(1, 4, 2, 8))
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_deltarule_bwd(z(1, 4, 2, 8), z(1, 4, 2, 8), z(1, 4, 2, 8), z(1, 4, 2, 8))
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_deltarule_update(z(1, 2, 8, 8), z(1, 2, 8), z(1, 2, 8), z(1, 2, 8))
    with pytest.raises(ValueError, match="q must be"):
        ssm.ssm_deltarule_fwd(z(4, 2, 8), z(4, 2, 8), z(4, 2, 8))
    with pytest.raises(ValueError, match="v must be"):
        ssm.ssm_deltarule_update(z(1, 2, 8, 8), z(1, 2, 8), z(1, 2, 8), z(1, 2, 8, 1))


@pytest.mark.gpu
def test_binding_on_the_gpu():
    import torch

    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    q, v = z(1, 4, 2, 8), z(1, 4, 4, 8)
    for kw, err, match in ((dict(beta=z(1, 4, 2)), ValueError, "beta has shape"), (dict(beta=z(1, 4, 4).bfloat16()), TypeError, "beta has dtype"),
                           (dict(beta=z(1, 4, 4).cpu()), ValueError, "beta is on"), (dict(beta=1.0), TypeError, "beta must be a torch.Tensor"),
                           (dict(beta=z(1, 4, 8)[..., ::2]), ValueError, "beta must be contiguous"), (dict(g=z(1, 4, 3)), ValueError, "g has shape"),
                           (dict(lengths=z(1)), TypeError, "lengths has dtype"), (dict(initial_state=z(1, 4, 8, 7)), ValueError, "initial_state has shape")):
        with pytest.raises(err, match=match):
            ssm.ssm_deltarule_fwd(q, q, v, **kw)
        with pytest.raises(err, match=match):
            ssm.ssm_deltarule_bwd(q, q, v, v, **kw)
    with pytest.raises(ValueError, match="must be a multiple"):
        ssm.ssm_deltarule_fwd(q, q, z(1, 4, 3, 8))
    S = z(1, 4, 8, 8)
    with pytest.raises(ValueError, match="initial_state must not be"):
        ssm.ssm_deltarule_fwd(q, q, v, initial_state=S, last_state=S)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.ssm_deltarule_fwd(q.half(), q.half(), v.half())
    with pytest.raises(ssm.SSMError):
        ssm.ssm_deltarule_fwd(z(1, 4, 2, 129), z(1, 4, 2, 129), v)
