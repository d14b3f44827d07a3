"""The gated delta rule's backward where one workgroup takes several heads of a group one after the other: all of them or some
(whose sums then are added), heads to 64 and above, one pass over the values or several, whole pieces or not.

Batch rows and groups of heads are independent, so some of them are held to the float64 reference, with the bounds of
tests/deltarule_ref.py, up to their length; all of them to the same call on one row alone, where every head has a workgroup of
its own, within both calls' bounds."""
import pytest

from tests import deltarule_plan as plan
from tests.gpu_common import say
from tests.test_gpu_deltarule import bwd, make

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dbeta", "dg", "d_initial_state")


def part(x, row, group, n):
    """One batch row's group of heads, of its first n tokens."""
    H, G = x["v"].shape[2], x["q"].shape[2]
    hs = slice(group * (H // G), (group + 1) * (H // G))
    out = dict(x, lengths=None)
    for k in ("q", "k"):
        out[k] = x[k][row:row + 1, :n, group:group + 1]
    for k in ("v", "dy", "beta", "g"):
        out[k] = None if x[k] is None else x[k][row:row + 1, :n, hs]
    for k in ("initial_state", "d_last_state"):
        out[k] = None if x[k] is None else x[k][row:row + 1, hs]
    out["A"] = None if x["A"] is None else x["A"][hs]
    return out


def part_of(name, t, x, row, group, n):
    H, G = x["v"].shape[2], x["q"].shape[2]
    hs = slice(group * (H // G), (group + 1) * (H // G))
    if name in ("dq", "dk"):
        return t[row:row + 1, :n, group:group + 1]
    if name == "d_initial_state":
        return t[row:row + 1, hs]
    return t[row:row + 1, :n, hs]


CASES = [  # b, L of bf16, H, G, Dk, Dv, heads of a workgroup
    (16, 1000, 16, 4, 128, 128, 4), (8, 1050, 16, 4, 128, 72, 2), (16, 1000, 16, 4, 72, 128, 4), (8, 1050, 16, 4, 100, 127, 2),
    (8, 1050, 16, 4, 64, 72, 2), (16, 1000, 16, 4, 33, 40, 4), (11, 1100, 18, 3, 48, 68, 3), (16, 700, 36, 4, 128, 33, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,L,H,G,Dk,Dv,together", CASES)
def test_heads_one_after_the_other(b, L, H, G, Dk, Dv, together, dtype):
    import torch

    from tests import deltarule_ref as ref

    L = L if dtype == "bf16" else L // 2
    assert plan.heads_together(b, L, H, G, dtype) == together
    assert plan.heads_together(1, L, H, G, dtype) == 1
    lengths = [L, 0, 1, 65, 130] + [L - 7 * i for i in range(5, b)]
    x = make(b=b, L=L, H=H, G=G, Dk=Dk, Dv=Dv, dtype=dtype, seed=L + Dk, lengths=lengths, fixed=True, rate=0.05)
    what = f"deltarule shared b={b} L={L} H={H} G={G} Dk={Dk} Dv={Dv} {dtype}"
    say(what)
    d = bwd(x)
    again = bwd(x)
    torch.cuda.synchronize()
    for k in GRADS:
        assert torch.equal(d[k], again[k]), k
    del again
    spread = {}
    for row, group in ((4, 0), (3, G - 1), (2, 1)):
        n = lengths[row]
        sub = part(x, row, group, n)
        want, V = ref.backward(sub)
        for k in GRADS:
            spread[k] = max(spread.get(k, 0.0), (V[k].sum() / want[k].square().sum()).item() ** 0.5) if n > 1 else spread[k]
            ref.within(part_of(k, d[k], x, row, group, n), want[k], V[k], k, sub, f"{what} row {row} group {group}")
    for row in range(b):
        for k in GRADS[:-1]:
            assert (d[k][row, lengths[row]:] == 0).all(), k
    assert torch.equal(d["d_initial_state"][1], x["d_last_state"][1])
    # whole rows, in the norm: both results round once, and both have the arithmetic's error, whose V is to the values as in
    # the rows above
    say(what + ", a row alone")
    for row in (0, b - 1):
        one = bwd({k: t[row:row + 1] if isinstance(t, torch.Tensor) and k != "A" else t for k, t in x.items()})
        torch.cuda.synchronize()
        for k in GRADS:
            got, want = d[k][row].double(), one[k][0].double()
            unit = 2.0 ** -24 * ref.terms(x) ** 0.5
            half = ref.HALF[d[k].dtype]
            if d[k].dtype == torch.bfloat16:
                unit += 4 * 2.0 ** -16
            rel = (got - want).norm().item() / want.norm().item()
            bound = 2 * (half + ref.SIGMAS * unit * spread[k])
            print(f"[deltarule] {what}: {k} of row {row} off by {rel:.2e} of its norm (bound {bound:.1e})", flush=True)
            assert rel <= bound, k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_gates_or_strengths(dtype):
    import torch

    from tests import deltarule_ref as ref

    b, L, H, G, Dk, Dv = 16, 1000 if dtype == "bf16" else 500, 16, 4, 96, 40
    assert plan.heads_together(b, L, H, G, dtype) == 4
    x = make(b=b, L=L, H=H, G=G, Dk=Dk, Dv=Dv, dtype=dtype, seed=2, gate=False, beta=None, init=False, lengths=[100] * b)
    say(f"deltarule shared, no gate and no beta {dtype}")
    d = bwd(x)
    torch.cuda.synchronize()
    assert d["dg"] is None and d["dbeta"] is None and d["d_initial_state"] is None
    sub = part(x, 9, 2, 100)
    want, V = ref.backward(sub)
    for k in ("dq", "dk", "dv"):
        ref.within(part_of(k, d[k], x, 9, 2, 100), want[k], V[k], k, sub, f"no gate, no beta {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_head_stays_in_its_group(dtype):
    """What is not finite in one head of a workgroup does not come into another one's own gradients, nor into another group's."""
    import torch

    b, L, H, G = 16, 1000 if dtype == "bf16" else 500, 16, 4
    assert plan.heads_together(b, L, H, G, dtype) == 4
    x = make(b=b, L=L, H=H, G=G, Dk=72, Dv=40, dtype=dtype, seed=3, lengths=[200] * b)
    say(f"deltarule shared, a bad head {dtype}")
    d0 = bwd(x)
    for name in ("v", "dy", "beta", "g"):
        z = dict(x, **{name: x[name].clone()})
        z[name][(3, 70, 5) if name in ("beta", "g") else (3, 70, 5, 0)] = float("nan")
        d = bwd(z)
        torch.cuda.synchronize()
        heads = [h for h in range(H) if h != 5]
        for k in ("dv", "dbeta", "dg"):
            assert torch.equal(d[k][:, :, heads], d0[k][:, :, heads]), (name, k)
        for k in ("dq", "dk"):
            assert torch.equal(d[k][:, :, [0, 2, 3]], d0[k][:, :, [0, 2, 3]]), (name, k)
        rows = [i for i in range(b) if i != 3]
        for k in GRADS:
            assert torch.equal(d[k][rows], d0[k][rows]), (name, k)
        assert not torch.isfinite(d["dk"][3, :200, 1]).all(), name
