"""Sequences that are cut into segments, and their segments' states into parts, with decays so slow that the states that
cross the cuts carry the outputs: against float64 on some of the heads, in the bounds of tests/linattn_ref.py,
tests/test_gpu_linattn_accuracy.py and tests/linattn_bounds.py."""
import pytest

from tests import linattn_bounds as bounds
from tests import linattn_ref as ref
from tests.gpu_common import say
from tests.test_gpu_linattn import bwd, fwd, make
from tests.test_gpu_linattn_accuracy import near

pytestmark = pytest.mark.gpu
F32_STATE = "last_state", "d_initial_state"


def some_heads(x, groups):
    """The inputs of the heads of some groups, alone."""
    H, G = x["v"].shape[2], x["q"].shape[2]
    heads = [g * (H // G) + i for g in groups for i in range(H // G)]
    z = dict(x)
    for k in ("q", "k"):
        z[k] = x[k][:, :, groups].contiguous()
    for k in ("v", "dy", "g"):
        z[k] = None if x[k] is None else x[k][:, :, heads].contiguous()
    z["A"] = None if x["A"] is None else x["A"][heads].contiguous()
    for k in ("initial_state", "d_last_state"):
        z[k] = None if x[k] is None else x[k][:, heads].contiguous()
    return z, heads


def check(x, dtype, what, segs_fwd, segs_bwd, groups):
    """Both directions; (segments, parts) are as the test means them to be."""
    import torch

    b, L, H, _ = x["v"].shape
    for backward, want in ((False, segs_fwd), (True, segs_bwd)):
        segs, parts, _ = bounds.cut(b, L, H, dtype, backward)
        assert (segs, parts) == want, (backward, segs, parts)
        assert bounds.parts_of(b, L, H, dtype, backward) == (segs - 1) * parts
    say(what)
    y, last = fwd(x)
    torch.cuda.synchronize()
    say(what + ", backward")
    d = bwd(x)
    torch.cuda.synchronize()
    z, heads = some_heads(x, groups)
    got = {"y": y[:, :, heads], "last_state": last[:, heads], "dq": d["dq"][:, :, groups], "dk": d["dk"][:, :, groups],
           "dv": d["dv"][:, :, heads]}
    if x["g"] is not None:
        got["dg"] = d["dg"][:, :, heads]
    if x["initial_state"] is not None:
        got["d_initial_state"] = d["d_initial_state"][:, heads]
    want, mag = {**ref.forward(z), **ref.backward(z)}, {**ref.forward(z, absolute=True), **ref.backward(z, absolute=True)}
    for name, t in got.items():
        ref.within(t, want[name], mag[name], name, z, what)
        if name in F32_STATE:
            over = bounds.state_over(t, want[name], z, name)
        elif name == "dg":
            over = bounds.dg_over(t, want[name], bounds.spread(z), z)
        else:
            if dtype == "bf16":
                near(t, want[name], mag[name], name, z, what)
            continue
        print(f"[cut] {what}: {name} at {over:.3f} of its bound", flush=True)
        assert over <= 1.0, f"{what}: {name} is {over:.3f} times its bound"


# (segments, parts) of forward and backward follow the name; a chunk is 64 tokens, in float 32
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128), (33, 70), (100, 127)])
def test_widths(Dk, Dv):
    x = make(b=1, L=1100, H=40, G=20, Dk=Dk, Dv=Dv, dtype="bf16", rate=1e-3, seed=Dk + Dv)
    check(x, "bf16", f"linattn cut Dk={Dk} Dv={Dv} bf16", (4, 1), (2, 2), [0, 13, 19])


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128), (33, 70)])
def test_widths_float(Dk, Dv):
    x = make(b=1, L=700, H=40, G=40, Dk=Dk, Dv=Dv, dtype="f32", rate=1e-3, seed=Dk + Dv)
    check(x, "f32", f"linattn cut Dk={Dk} Dv={Dv} f32", (5, 1), (2, 2), [0, 13, 39])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts_of_both_directions(dtype):
    """Segments of several parts forwards, over many heads; the backward is uncut there."""
    L = 1600 if dtype == "bf16" else 800
    x = make(b=1, L=L, H=100, G=100, Dk=64, Dv=40, dtype=dtype, rate=1e-3, seed=5)
    check(x, dtype, f"linattn parts forwards {dtype}", (2, 3), (1, 1), [0, 57, 99])
    x = make(b=1, L=L, H=25, G=25, Dk=40, Dv=64, dtype=dtype, rate=1e-3, seed=6)
    check(x, dtype, f"linattn parts backwards {dtype}", (5, 1), (3, 2), [0, 11, 24])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_rows(dtype):
    import torch

    L = 1100 if dtype == "bf16" else 700
    x = make(b=1, L=L, H=40, G=40, Dk=64, Dv=64, dtype=dtype, rate=1e-3, seed=7)
    for k in ("q", "k", "v", "dy"):
        buf = torch.empty(x[k].numel() + 1, dtype=x[k].dtype, device="cuda")
        buf[1:] = x[k].reshape(-1)
        x[k] = buf[1:].view(x[k].shape)
    check(x, dtype, f"linattn cut unaligned {dtype}", (4 if dtype == "bf16" else 5, 1), (2, 2), [0, 20, 39])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_resets_and_fixed_decays(dtype):
    """Rows that end inside a segment, at its end, before it and nowhere; resets on both sides of a cut; a head's own decay."""
    import math

    import torch

    L = 1100 if dtype == "bf16" else 550
    unit = 64 if dtype == "bf16" else 32
    per = bounds.cut(4, L, 10, dtype, True)
    edge = per[1] * per[2] * unit  # the backward's cut
    lengths = [edge - 3, edge, L, 1]
    x = make(b=4, L=L, H=10, G=5, Dk=64, Dv=48, dtype=dtype, rate=1e-3, seed=8, lengths=lengths)
    check(x, dtype, f"linattn cut lengths {dtype}", (4, 1), (2, 2), [0, 4])
    x["lengths"] = None
    for t in (edge - 1, edge, edge + 40):
        x["g"][:, t] = -math.inf
    check(x, dtype, f"linattn cut resets {dtype}", (4, 1), (2, 2), [1])
    x["g"], x["A"] = None, torch.linspace(-2e-3, 0.0, 10).cuda()
    check(x, dtype, f"linattn cut fixed decay {dtype}", (4, 1), (2, 2), [0, 2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,rate", [(513, 0.1), (1500, 0.01), (200, 6.0), (200, 1e-4)])
def test_gates_are_right_to_their_last_roundings(L, rate, dtype):
    """The lengths and decays at which an elementwise bound of dg says little, cut and uncut."""
    import torch

    x = make(b=1, L=L, H=2, G=1 if L == 1500 else 2, Dk=64, Dv=48, dtype=dtype, rate=rate, seed=L)
    say(f"linattn dg L={L} rate={rate} {dtype}")
    d = bwd(x)
    torch.cuda.synchronize()
    over = bounds.dg_over(d["dg"], ref.backward(x)["dg"], bounds.spread(x), x)
    print(f"[cut] dg L={L} rate={rate} {dtype}: {over:.3f} of its bound", flush=True)
    assert over <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [64, 200, 1500])
def test_states_keep_their_bits(L, dtype):
    """States that are outputs hold all bits of a float: the third bf16 part of what is written into them is there."""
    import torch

    x = make(b=1, L=L, H=2, G=1, Dk=64, Dv=48, dtype=dtype, rate=0.01, seed=L)
    say(f"linattn states L={L} {dtype}")
    _, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    for name, got, f in (("last_state", last, ref.forward), ("d_initial_state", d["d_initial_state"], ref.backward)):
        over = bounds.state_over(got, f(x)[name], x, name)
        print(f"[cut] {name} L={L} {dtype}: {over:.3f} of its bound", flush=True)
        assert over <= 1.0, (name, over)
