"""Host-side checks of the entry points of the norms around a block: no GPU needed.  Refusals come back as the documented
ssm_status before anything is enqueued, the size limits are where the header says, and the binding names the argument that
does not fit."""
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
    a = dict(x=FAKE, w1=None, z=None, scale=None, residual=None, w2=None, eps=1e-5, norms=3, h=FAKE, n=FAKE, r1=None, r2=None,
             rows=4, H=1, W=64, dtype=1, rdtype=1, stream=None)
    a.update(kw)
    return lib.ssm_blocknorm_fwd(*a.values())


def bwd(lib, **kw):
    a = dict(x=FAKE, w1=None, z=None, scale=None, residual=None, w2=None, norms=3, r1=FAKE, r2=FAKE, dh=FAKE, dn=FAKE, dx=FAKE,
             dz=None, dres=None, dw1=None, dscale=None, dw2=None, rows=4, H=1, W=64, dtype=1, rdtype=1, ws=None, bytes=0, stream=None)
    a.update(kw)
    return lib.ssm_blocknorm_bwd(*a.values())


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    for s in (dict(rows=-1), dict(H=-1), dict(W=0), dict(W=16385), dict(W=-5), dict(rows=1 << 40), dict(rows=1 << 31),
              dict(H=1 << 30), dict(norms=0), dict(norms=4), dict(norms=-1)):
        assert call(lib, **s) == DIM, s
    for s in (dict(dtype=7), dict(rdtype=2), dict(dtype=0, rdtype=1), dict(dtype=-1)):
        assert call(lib, **s) == DTYPE, s
    for n in ("x", "n") if call is fwd else ("x", "r1", "r2", "dn", "dx"):
        assert call(lib, **{n: None}) == NULL, n
    first = "h" if call is fwd else "dh"
    assert call(lib, norms=1, **{first: None}) == NULL
    assert call(lib, x=FAKE + 1) == ALIGN and call(lib, x=FAKE + 2, dtype=0, rdtype=0) == ALIGN
    for n in ("w1", "scale", "w2", "r1", "r2"):
        assert call(lib, **{n: FAKE + 2}) == ALIGN, n
    assert call(lib, residual=FAKE + 2, rdtype=0) == ALIGN and call(lib, z=FAKE + 1) in (ALIGN, NULL)
    assert call(lib, H=0, x=None) == OK


@pytest.mark.parametrize("call", [fwd, bwd])
def test_documented_limits(lib, call):
    """Just inside, only a missing pointer is refused; just outside, the size is."""
    for inside, outside in ((dict(rows=2 ** 31 - 1), dict(rows=2 ** 31)), (dict(rows=2 ** 21, H=2 ** 9), dict(rows=2 ** 21, H=2 ** 10)),
                            (dict(W=16384), dict(W=16385)), (dict(H=2 ** 21, W=127), dict(H=2 ** 21, W=128)),
                            (dict(H=2 ** 21, W=1), dict(H=2 ** 21 + 1, W=1)), (dict(H=2 ** 14 - 1, W=2 ** 14), dict(H=2 ** 14, W=2 ** 14))):
        assert call(lib, **dict(inside, x=None)) == NULL, inside
        assert call(lib, **dict(outside, x=None)) == DIM, outside


def test_more(lib):
    assert fwd(lib, eps=-1.0) == DIM and fwd(lib, eps=float("nan")) == DIM
    assert fwd(lib, rows=0, x=None, h=None, n=None) == OK
    assert bwd(lib, z=FAKE) == NULL and bwd(lib, z=FAKE, dz=FAKE + 1) == ALIGN
    assert bwd(lib, dw1=FAKE, ws=FAKE, bytes=4) == SCRATCH and bwd(lib, dw1=FAKE, ws=FAKE, bytes=-1) == SCRATCH
    assert bwd(lib, dscale=FAKE + 2) == ALIGN and bwd(lib, dres=FAKE + 2, rdtype=0) == ALIGN
    need = ssm.ssm_blocknorm_workspace(4, 1, 64)
    assert need > 0 and bwd(lib, dw2=FAKE, ws=FAKE + 128, bytes=need) == ALIGN
    assert bwd(lib, rows=0, x=None, r1=None, r2=None, dh=None, dn=None, dx=None) == OK
    assert ssm.ssm_blocknorm_workspace(0, 1, 64) == 0 and ssm.ssm_blocknorm_workspace(9, 2, 64, "bf16", "f32") > 0
    for bad in (dict(rows=4, H=1, W=0), dict(rows=4, H=1, W=8, dtype="f32", residual_dtype="bf16"), dict(rows=-1, H=1, W=8)):
        with pytest.raises(ssm.SSMError):
            ssm.ssm_blocknorm_workspace(**bad)


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    if not os.path.exists(ssm.library_path()):
        pytest.skip("libssm.so not built")
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_blocknorm_fwd(z)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_blocknorm_bwd(z, z[:, 0], z[:, 0], z, z)
    with pytest.raises(ValueError, match="norms must be"):
        ssm.ssm_blocknorm_fwd(z, norms="none")
    with pytest.raises(ValueError, match="post_weight is given"):
        ssm.ssm_blocknorm_fwd(z, post_weight=z[0], norms="pre")
    with pytest.raises(ValueError, match="pre_weight is given"):
        ssm.ssm_blocknorm_fwd(z, pre_weight=z[0], norms="post")
    with pytest.raises(ValueError, match="x must be"):
        ssm.ssm_blocknorm_fwd(None)


@pytest.mark.gpu
def test_binding_on_the_gpu():
    import torch

    z = torch.zeros(4, 2, 8, device="cuda")
    for kw, err, match in ((dict(z=z[:2]), ValueError, "z has shape"), (dict(z=z.bfloat16()), TypeError, "z has dtype"),
                           (dict(residual=z.bfloat16()), TypeError, "residual has dtype"), (dict(residual=2.0), TypeError, "residual must be"),
                           (dict(scale=torch.zeros(2, 8)), ValueError, "scale is on"), (dict(scale=torch.zeros(3, 8, device="cuda")), ValueError, "do not fit"),
                           (dict(scale=torch.zeros(8, device="cuda"), post_weight=torch.zeros(2, 8, device="cuda")), ValueError, "scale has shape")):
        with pytest.raises(err, match=match):
            ssm.ssm_blocknorm_fwd(z, **kw)
    stat = torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError, match="rstd_post is required"):
        ssm.ssm_blocknorm_bwd(z, None, stat, z, z)
    with pytest.raises(ValueError, match="dh is required"):
        ssm.ssm_blocknorm_bwd(z, stat, None, None, None, norms="post")
    with pytest.raises(ValueError, match="n is given"):
        ssm.ssm_blocknorm_fwd(z, norms="post", n=z.clone())
