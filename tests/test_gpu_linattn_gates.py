"""The gradient of the gates where documents follow each other in a row: a token whose decay is zero in float drops the
state, so nothing of a document may come into the gradients of the one before it."""
import math

import pytest

from tests.gpu_common import say
from tests.test_gpu_linattn import bwd, make

pytestmark = pytest.mark.gpu


def documents(L, starts, dtype, seed, lengths=None, fixed=0.0, value=-math.inf):
    """A batch of two rows with resets at ``starts``; with ``fixed`` a part of their log decay is the head's own."""
    import torch

    x = make(b=2, L=L, H=18, G=9, Dk=32, Dv=40, dtype=dtype, seed=seed, rate=0.05, lengths=lengths)
    if fixed:
        x["A"] = torch.full((18,), fixed, device="cuda")
        x["g"] -= fixed  # the log decays of the other tokens as before, but for a rounding
    for t in starts:
        x["g"][:, t] = value
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,starts", [(90, [1, 40, 41]), (300, [0, 100, 260]), (600, [255, 256]), (1300, [17, 900]), (1100, [300, 301, 700])])
def test_a_document_alone(L, starts, dtype):
    """Whatever the later documents hold, the gate gradients of the earlier ones keep every bit; at a reset they are zero."""
    import torch

    x = documents(L, starts, dtype, seed=L)
    say(f"linattn gates L={L} {starts} {dtype}")
    d0 = bwd(x)
    torch.cuda.synchronize()
    assert (d0["dg"][:, starts] == 0).all()
    gen = torch.Generator().manual_seed(7)
    for t in starts:
        z = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
        for k in ("q", "k", "v", "dy"):
            z[k][:, t:] = (100 * torch.randn(z[k][:, t:].shape, generator=gen)).to(z[k].dtype).cuda()
        z["d_last_state"] = 1e4 * z["d_last_state"]
        d = bwd(z)
        torch.cuda.synchronize()
        assert torch.equal(d["dg"][:, :t + 1], d0["dg"][:, :t + 1]), t
        assert not torch.equal(d["dg"][:, t + 1:], d0["dg"][:, t + 1:]) or t + 1 in starts
        for name in ("k", "v"):  # a value that is not finite too
            z = dict(x, **{name: x[name].clone()})
            z[name][:, min(t + 2, L - 1), 3, 1] = float("nan")
            d = bwd(z)
            torch.cuda.synchronize()
            assert torch.equal(d["dg"][:, :t + 1], d0["dg"][:, :t + 1]), (name, t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_by_both_decays_and_behind_the_length(dtype):
    """g and A together make a reset; a token behind the row's length makes none, whatever its gate holds."""
    import torch

    say(f"linattn gates of both decays {dtype}")
    x = documents(500, [120, 300], dtype, seed=3, fixed=-60.0, value=-60.0)
    d = bwd(x)
    torch.cuda.synchronize()
    assert (d["dg"][:, [120, 300]] == 0).all() and torch.isfinite(d["dg"]).all()
    x = documents(500, [], dtype, seed=4, lengths=[300, 431])
    d0 = bwd(x)
    x["g"][0, 300:] = -math.inf
    x["g"][1, 431:] = float("nan")
    d = bwd(x)
    torch.cuda.synchronize()
    assert torch.equal(d["dg"], d0["dg"])


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (33, 70)])
def test_the_last_states_part_of_float_gates(Dk, Dv):
    """Without decays, keys and dy every dg is <d_last_state, initial_state>, a sum of up to 16384 products that is part
    of the dg of every token: the products are exact in float64 and the sum is off by 2^-52 of its terms' sizes, so
    dg is off by its own rounding."""
    import torch

    x = make(b=2, L=70, H=3, G=3, Dk=Dk, Dv=Dv, dtype="f32", seed=Dk)
    for k in ("k", "dy", "g"):
        x[k].zero_()
    say(f"linattn end of the gates Dk={Dk} Dv={Dv}")
    d = bwd(x)
    torch.cuda.synchronize()
    terms = x["d_last_state"].double() * x["initial_state"].double()
    want = terms.sum((-1, -2))[:, None].expand(2, 70, 3)
    tol = want.abs() * 2.0 ** -24 + terms.abs().sum((-1, -2))[:, None] * Dk * Dv * 2.0 ** -52
    assert ((d["dg"].double() - want).abs() <= tol * 1.01).all(), ((d["dg"].double() - want).abs() / tol).max()
