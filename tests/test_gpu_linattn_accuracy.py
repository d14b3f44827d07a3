"""How near linear attention's outputs are to float64, in bounds that one lost rounding breaks.

Beside those of tests/linattn_ref.py, whose magnitudes and counts of roundings are used here:

* y, dq, dk, dv of bf16 tensors: an operand that is not given in bf16 (the mixing matrix, the state that is read, the
  values that are written into a state) is taken in two bf16 parts at least.  The first is off by 2^-8 of it at most, the
  second by 2^-8 of that: 2^-16.  A product goes through one such operand inside its chunk, through two (written and
  read) beyond it: 2^-15 of the magnitude.  Then the output's own rounding, 2^-8 of the value.
"""
import pytest

from tests import linattn_ref as ref
from tests.gpu_common import say
from tests.test_gpu_linattn import bwd, fwd, make

pytestmark = pytest.mark.gpu
PARTS = 2.0 ** -15


def near(got, want, mag, name, x, what):
    """The elementwise bound above (bf16), of an output in the streamed type."""
    tol = mag * (PARTS + 2 * ref.terms(x) * 2.0 ** -24) + want.abs() * 2.0 ** -8
    over = ((got.detach().cpu().to(ref.F64) - want).abs() / (tol * 1.01 + 1e-37)).max().item()
    print(f"[accuracy] {what}: {name} at {over:.3f} of its bound", flush=True)
    assert over <= 1.0, f"{what}: {name} is {over:.3f} times its bound"


SIZES = [dict(L=200, H=4, G=2, Dk=64, Dv=64), dict(L=150, H=2, G=2, Dk=64, Dv=128), dict(L=150, H=2, G=1, Dk=128, Dv=64),
         dict(L=130, H=2, G=2, Dk=128, Dv=128), dict(L=140, H=3, G=3, Dk=40, Dv=24), dict(L=97, H=2, G=2, Dk=33, Dv=70),
         dict(L=130, H=2, G=2, Dk=100, Dv=127), dict(L=1500, H=2, G=1, Dk=64, Dv=48, rate=0.01)]


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_outputs_are_rounded_once(size, gate):
    """Without a gate too: the sweeps that need no dots are other kernels."""
    import torch

    x = make(b=1, seed=31, gate=gate, fixed=not gate, **size)
    what = f"linattn {size} gate={gate}"
    say(what)
    y, _ = fwd(x)
    torch.cuda.synchronize()
    near(y, ref.forward(x)["y"], ref.forward(x, absolute=True)["y"], "y", x, what)
    d = bwd(x)
    torch.cuda.synchronize()
    want, mag = ref.backward(x), ref.backward(x, absolute=True)
    for name in ("dq", "dk", "dv"):
        near(d[name], want[name], mag[name], name, x, what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [200, 1500])
def test_what_else_is_asked_for_changes_no_bit(L, dtype):
    """y is the same with and without last_state, dv with and without the gradient of an initial state of zero."""
    import torch

    x = make(b=1, L=L, H=2, G=1, Dk=64, Dv=48, dtype=dtype, rate=0.01, seed=32)
    x["d_last_state"] = None
    say(f"linattn optional outputs L={L} {dtype}")
    y, _ = fwd(x)
    alone, none = fwd(x, return_last_state=False)
    assert none is None and torch.equal(y, alone)
    zero = torch.zeros_like(x["initial_state"])
    d0, d = bwd(dict(x, initial_state=zero)), bwd(dict(x, initial_state=None))
    torch.cuda.synchronize()
    for name in ("dq", "dk", "dv", "dg"):
        assert torch.equal(d0[name], d[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("size", [dict(Dk=40, Dv=72), dict(Dk=64, Dv=64), dict(Dk=128, Dv=128), dict(L=1500, H=2, G=2, Dk=64, Dv=64)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_what_is_not_finite_reaches_what_reads_it(size, bad, dtype):
    """One value that is not finite changes no bit of the outputs that do not read it by the definition: tokens before
    it (in the backward, of q and dy, those after), the other columns of v, other heads."""
    import torch

    x = make(**dict(dict(b=1, L=200, H=2, G=2, dtype=dtype, seed=21, rate=0.05), **size))
    x["d_last_state"] = None
    say(f"linattn {size} {bad} {dtype}")
    L = x["v"].shape[1]
    y0, _ = fwd(x)
    d0 = bwd(x)

    def same(a, b, what):
        assert torch.equal(a, b), what

    for t in (0, 40, 63, 64, 127, L - 1):
        for name in ("q", "k", "v", "dy"):
            z = dict(x, **{name: x[name].clone()})
            z[name][0, t, 1, 5] = bad
            at = (name, t)
            y, _ = fwd(z)
            d = bwd(z)
            torch.cuda.synchronize()
            same(y[:, :, 0], y0[:, :, 0], at)
            for n in d:
                if n == "d_initial_state":
                    same(d[n][:, 0], d0[n][:, 0], at)
                else:
                    same(d[n][:, :, 0], d0[n][:, :, 0], at)
            if name == "dy":
                same(y, y0, at)
            else:
                same(y[:, :t], y0[:, :t], at)
                assert not torch.isfinite(y[0, t, 1, 5 if name == "v" else 0])
            if name == "q":
                same(y[:, t + 1:], y0[:, t + 1:], at)
                same(d["dq"], d0["dq"], at)
            if name == "v":
                same(y[:, :, 1, :5], y0[:, :, 1, :5], at)
                same(y[:, :, 1, 6:], y0[:, :, 1, 6:], at)
                assert not torch.isfinite(y[0, t:, 1, 5]).any()
            if name in ("k", "v"):
                same(d["dq"][:, :t], d0["dq"][:, :t], at)
                assert not torch.isfinite(d["dq"][0, t:, 1, 5]).any()
                n, alone = ("dv", "dk") if name == "v" else ("dk", "dv")
                same(d[n], d0[n], at)  # read by no dv (of v), by no dk (of k) ...
                same(d[alone][:, :t], d0[alone][:, :t], at)  # ... and by its own token's dk, dv
                same(d[alone][:, t + 1:], d0[alone][:, t + 1:], at)
                same(d["d_initial_state"], d0["d_initial_state"], at)
            if name in ("q", "dy"):
                for n in ("dk", "dv", "dg"):
                    same(d[n][:, t + 1:], d0[n][:, t + 1:], (n, *at))
                assert not torch.isfinite(d["dk"][0, :t + 1, 1, 5]).any()
            if name == "dy":
                same(d["dq"][:, :t], d0["dq"][:, :t], at)
                same(d["dq"][:, t + 1:], d0["dq"][:, t + 1:], at)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate,L", [(0.4, 130), (1.2, 64)])
def test_states_that_grow(rate, L, dtype):
    """Positive log decays, which add up to some 20 and 60 over a chunk."""
    import torch

    x = make(b=1, L=L, H=2, G=2, Dk=40, Dv=64, dtype=dtype, seed=33, rate=-rate)
    assert (x["g"] >= 0).all()
    what = f"linattn growing {rate} {dtype}"
    say(what)
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    want, mag = {**ref.forward(x), **ref.backward(x)}, {**ref.forward(x, absolute=True), **ref.backward(x, absolute=True)}
    for name, t in {"y": y, "last_state": last, **d}.items():
        ref.within(t, want[name], mag[name], name, x, what)
