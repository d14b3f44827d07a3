"""The float64 reference of linear attention pinned on the CPU: against the closed form without a
recurrence, and its gradients against central differences of its forward."""
import pytest
import torch

from tests import linattn_ref as ref

F64 = torch.float64


def make(b=2, L=7, H=4, G=2, Dk=3, Dv=5, seed=0, lengths=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=F64)  # noqa: E731
    return {"q": n(b, L, G, Dk), "k": n(b, L, G, Dk), "v": n(b, L, H, Dv), "g": -n(b, L, H).abs(), "A": -n(H).abs(),
            "scale": 0.7, "lengths": lengths, "initial_state": n(b, H, Dk, Dv), "dy": n(b, L, H, Dv),
            "d_last_state": n(b, H, Dk, Dv)}


@pytest.mark.parametrize("lengths", [None, [7, 3], [0, 1]])
def test_forward_is_the_masked_product(lengths):
    x = make(lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    out = ref.forward(x)
    b, L, H, Dv = x["v"].shape
    for i in range(b):
        n = L if lengths is None else lengths[i]
        for h in range(H):
            q, k, v = x["q"][i, :n, h // 2], x["k"][i, :n, h // 2], x["v"][i, :n, h]
            c = (x["g"][i, :n, h] + x["A"][h]).cumsum(0)
            mask = torch.tril(torch.ones((n, n), dtype=F64)) * torch.exp(torch.tril(c[:, None] - c[None]))
            y = 0.7 * ((q @ k.T) * mask @ v + torch.exp(c)[:, None] * (q @ x["initial_state"][i, h]))
            assert torch.allclose(out["y"][i, :n, h], y, rtol=1e-12, atol=1e-12)
            assert (out["y"][i, n:, h] == 0).all()


@pytest.mark.parametrize("lengths", [None, [7, 3], [0, 1]])
def test_gradients_against_differences(lengths):
    x = make(seed=3, lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    grads = ref.backward(x)

    def loss(z):
        out = ref.forward(z)
        return float((out["y"] * z["dy"]).sum() + (out["last_state"] * z["d_last_state"]).sum())

    rng = torch.Generator().manual_seed(1)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("initial_state", "d_initial_state")):
        for _ in range(3):
            way = torch.randn(x[name].shape, generator=rng, dtype=F64)
            e = 1e-5
            up, down = dict(x), dict(x)
            up[name], down[name] = x[name] + e * way, x[name] - e * way
            want = (loss(up) - loss(down)) / (2 * e)
            got = float((grads[grad] * way).sum())
            assert abs(got - want) <= 1e-7 * (1 + abs(want)), (name, got, want)


def test_magnitudes_bound_the_values():
    x = make(seed=5)
    for f in (ref.forward, ref.backward):
        val, mag = f(x), f(x, absolute=True)
        for k in val:
            assert (val[k].abs() <= mag[k] * (1 + 1e-12)).all(), k
