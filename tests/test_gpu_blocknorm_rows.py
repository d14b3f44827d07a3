"""The norms around a block on calls of so many rows that every group of threads walks several: one norm alone or both, with
rows of a wave, of a few waves and of more than 1024 vectors.

A row's results do not depend on the rows around it, so they are bit for bit those of calls so small that a group has one row
(which tests/test_gpu_blocknorm.py holds to float64).  The parameters' gradients are held to float64.  Bound: the values of a
term come from sums over a row, at most 16 elements one after the other in a thread, 6 steps in a wave and 16 waves, four of
them along the chain; a term is one of ``rows / n`` in its group, of n / 16 and 24 more in the sum of the n groups' parts, and
each step is off by 2^-24 of the sum of the terms' magnitudes at most.  A row that is left out or taken twice is 1 / rows
of that sum on average, and is over the bound in the columns where it is some times more.
"""
import pytest

from tests.gpu_common import say
from tests.test_gpu_blocknorm import FORMS, check, close, definition, make as make_small

pytestmark = pytest.mark.gpu
EPS = 1e-5


def slices(W, H, dtype, forward):
    """Rows in flight of one head: workgroups by groups of threads in each (as csrc/ssm_blocknorm.hip deals them)."""
    vectors = -(-W // (8 if dtype == "bf16" else 4))
    tpr = next((t for t in (8, 16, 32, 64, 128) if vectors <= t), 256)
    groups = 256 // tpr if tpr <= 128 else 1
    blocks = 8192 if forward else 512 if tpr > 64 else 768
    return -(-blocks * groups // H)


def make(rows, H, W, dtype, form, seed):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    io = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    res = {"none": None, "same": io, "f32": torch.float32}[form["residual"]]
    shape, par = ((rows, W), (W,)) if H == 1 else ((rows, H, W), (H, W))
    x = {"x": (1.5 * n(*shape)).to(io), "z": (2 * n(*shape)).to(io) if form["gate"] else None,
         "residual": None if res is None else (2 * n(*shape)).to(res),
         "post_weight": 1 + 0.3 * n(*par) if form["post"] else None, "pre_weight": 1 + 0.3 * n(*par) if form["pre"] else None,
         "scale": 0.5 + 0.2 * n(*par) if form.get("scale", True) else None,
         "norms": "both" if form["post"] and form["pre"] else "post" if form["post"] else "pre"}
    return x, {"dh": n(*shape).to(res or io), "dn": n(*shape).to(io) if form["pre"] else None}


def both(x, d, H):
    """All results of the forward and the backward by name."""
    import selective_state_space_35_amd as ssm

    heads = None if H == 1 else H
    given = {k: x[k] for k in x if k != "x"}
    h, n, r1, r2 = ssm.ssm_blocknorm_fwd(x["x"], **given, eps=EPS, heads=heads)
    return {"h": h, "n": n, "rstd_post": r1, "rstd_pre": r2, **ssm.ssm_blocknorm_bwd(x["x"], r1, r2, **d, **given, heads=heads)}


PARAMS = ("dpost_weight", "dscale", "dpre_weight")
WALKS = [dict(post=False, pre=True, gate=False, residual="same", scale=False), dict(post=False, pre=True, gate=True, residual="f32"),
         dict(post=True, pre=False, gate=True, residual="none", scale=False), dict(post=True, pre=False, gate=False, residual="same"),
         dict(post=True, pre=True, gate=False, residual="same"), dict(post=True, pre=True, gate=True, residual="f32")]


def walk(rows, H, W, dtype, form, what):
    import torch

    for forward in (True, False):
        n = slices(W, H, dtype, forward)
        assert rows > 2 * n and rows % n, (rows, n)
    few_rows = min(n, 512)  # of a call in which every group has one row at most
    say(what)
    x, d = make(rows, H, W, dtype, form, W + rows)
    got = both(x, d, H)
    again = both(x, d, H)
    torch.cuda.synchronize()
    for k, t in got.items():
        assert t is None or torch.equal(t, again[k]), f"{what}: {k} differs from run to run"
    del again
    say(what + ", by small calls")
    cut = lambda t, a: t[a:a + few_rows] if isinstance(t, torch.Tensor) and t.shape[0] == rows else t  # noqa: E731
    for a in range(0, rows, few_rows):
        few = both({k: t if k in ("post_weight", "pre_weight", "scale") else cut(t, a) for k, t in x.items()},
                   {k: cut(t, a) for k, t in d.items()}, H)
        for k, t in few.items():
            if t is not None and k not in PARAMS:
                assert torch.equal(t, got[k][a:a + few_rows]), f"{what}: {k} of rows {a} on"
    say(what + ", parameters")
    f64 = lambda t: t.double() if isinstance(t, torch.Tensor) else t  # noqa: E731
    ref = {k: f64(t) for k, t in x.items()}
    names = [k for k in ("post_weight", "scale", "pre_weight") if x[k] is not None]
    leaves = {k: ref[k].clone().requires_grad_() for k in names}
    wh, wn, _, w2 = definition({**ref, **leaves}, EPS)
    ((wh * f64(d["dh"])).sum() + (0 if wn is None else (wn * f64(d["dn"])).sum())).backward()
    wh = wh.detach()
    with torch.no_grad():  # magnitudes: the chain with every term positive
        a = lambda t: 1.0 if t is None else t.abs()  # noqa: E731
        u = wh if ref["residual"] is None else wh - ref["residual"]
        if ref["z"] is not None:
            u = u * (1 + ref["z"].abs())
        part = u.abs()
        e = f64(d["dh"]).abs()
        mags = {}
        if w2 is not None:
            hh = (part + (0.0 if ref["residual"] is None else ref["residual"].abs())) * w2.detach()[..., None]
            t = f64(d["dn"]).abs() * a(ref["pre_weight"])
            e = e + w2.detach()[..., None] * (t + hh * (t * hh).mean(-1, keepdim=True))
            mags["pre_weight"] = (f64(d["dn"]).abs() * hh).sum(0)
        mags["scale"] = (e * part / a(ref["scale"])).sum(0)
        if ref["post_weight"] is not None:
            mags["post_weight"] = (e * part / a(ref["post_weight"])).sum(0)
    n = slices(W, H, dtype, False)
    terms = 4 * (16 + 6 + 16) + -(-rows // n) + -(-n // 16) + 24
    for k in names:
        close(got["d" + k], leaves[k].grad.cpu(), mags[k].cpu(), 2.0 ** -24, terms, f"{what} d{k}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(WALKS)))
@pytest.mark.parametrize("bytes_of_a_row", [1024, 1040, 2304, 5120, 16400])
def test_rows_in_turn(bytes_of_a_row, form, dtype):
    """A wave's 64 vectors and one more, groups of three waves and of five, and more than 1024 vectors."""
    W = bytes_of_a_row // (2 if dtype == "bf16" else 4)
    walk(2 * max(slices(W, 1, dtype, True), 512) + 7, 1, W, dtype, WALKS[form], f"blocknorm rows W={W} form {form} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(WALKS)))
@pytest.mark.parametrize("H,W", [(24, 64), (3, 521), (7, 1537)])
def test_rows_of_heads_in_turn(H, W, form, dtype):
    walk(2 * slices(W, H, dtype, True) + 5, H, W, dtype, WALKS[form], f"blocknorm rows H={H} W={W} form {form} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("H,W", [(1, 520), (3, 1031), (1, 4104), (1, 8200)])
def test_forms_of_wide_rows(H, W, form, dtype):
    """The forms of tests/test_gpu_blocknorm.py at rows of several waves, against float64."""
    check(*make_small(rows=11, H=H, W=W, dtype=dtype, seed=form, **FORMS[form]), f"blocknorm form {form} H={H} W={W} {dtype}")
