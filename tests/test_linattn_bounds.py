"""The bounds of tests/linattn_bounds.py refuse what they are there to refuse, and the cut of a sequence is the one
that tests of it count on (CPU only)."""
import os

import pytest
import torch

import selective_state_space_35_amd as ssm
from tests import linattn_bounds as bounds
from tests import linattn_ref as ref


def make(L, G, Dv, rate, dtype, seed, H=2, Dk=64):
    gen = torch.Generator().manual_seed(seed)
    io = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = {"q": n(1, L, G, Dk), "k": n(1, L, G, Dk), "v": n(1, L, H, Dv), "dy": n(1, L, H, Dv), "g": -rate * n(1, L, H).abs()}
    x = {k: t.to(io) for k, t in x.items()}
    x.update(A=None, lengths=None, scale=Dk ** -0.5, initial_state=n(1, H, Dk, Dv), d_last_state=n(1, H, Dk, Dv))
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,G,Dv,rate", [(129, 2, 64, 0.1), (513, 2, 64, 0.1), (700, 1, 48, 0.01), (200, 2, 24, 6.0), (200, 2, 24, 1e-4)])
def test_the_bound_of_dg_refuses_lost_roundings(L, G, Dv, rate, dtype):
    x = make(L, G, Dv, rate, dtype, seed=L)
    io = x["v"].dtype
    H = x["v"].shape[2]
    z = dict(x, q=ref.heads(x["q"], H), k=ref.heads(x["k"], H))
    d = ref.backward(z)
    V = bounds.spread(x)
    assert bounds.dg_over(d["dg"].to(io), d["dg"], V, x) <= 1.0  # rounded once
    assert bounds.dg_over(torch.zeros_like(d["dg"]), d["dg"], V, x) > 20
    # from dq and dk as they are given out in bf16, with and without the token's product with itself
    end = (x["d_last_state"].to(ref.F64) * ref.forward(z)["last_state"]).sum((-1, -2))[:, None]
    vdy = (z["v"].to(ref.F64) * z["dy"].to(ref.F64)).sum(-1, keepdim=True) * x["scale"]
    for own in (1.0, 0.0):
        dq, dk = d["dq"] - (1 - own) * vdy * z["k"], d["dk"] - (1 - own) * vdy * z["q"]
        a = (z["q"] * dq.to(torch.bfloat16).to(ref.F64)).sum(-1) - (z["k"] * dk.to(torch.bfloat16).to(ref.F64)).sum(-1)
        got = (a.flip(1).cumsum(1).flip(1) + end).to(io)
        over = bounds.dg_over(got, d["dg"], V, x)
        print(f"[bounds] L={L} rate={rate} {dtype} own={own}: {over:.2f}")
        assert over > 1.25, (own, over)


@pytest.mark.parametrize("L", [64, 200, 700])
def test_the_bound_of_states_refuses_two_parts(L):
    """What is written into the state in two bf16 parts where it should be three: each value times its decay to the end."""
    x = make(L, 2, 48, 0.01, "bf16", seed=L)
    want = ref.forward(x)["last_state"]
    assert bounds.state_over(want.float(), want, x, "last_state") <= 1.0
    lg = x["g"].to(ref.F64).cumsum(1)
    w = (lg[:, -1:] - lg).exp()[..., None] * x["v"].to(ref.F64)  # [b, L, H, Dv]
    high = w.to(torch.bfloat16).to(ref.F64)
    parts = high + (w - high).to(torch.bfloat16).to(ref.F64)
    S = (x["k"].to(ref.F64)[..., None] * parts[..., None, :]).sum(1) + lg[:, -1].exp()[..., None, None] * x["initial_state"].to(ref.F64)
    over = bounds.state_over(S, want, x, "last_state")
    print(f"[bounds] L={L}: {over:.2f}")
    assert over > 1.25


def test_squares_are_the_sums_of_squares():
    """V against the definition: every product that a dg is made of, squared, one by one."""
    x = make(5, 1, 2, 0.3, "f32", 3, H=1, Dk=3)
    q, k, v, dy = (x[n][0, :, 0].to(ref.F64) for n in ("q", "k", "v", "dy"))
    g = x["g"][0, :, 0].to(ref.F64)
    S0, D0, s = x["initial_state"][0, 0].to(ref.F64), x["d_last_state"][0, 0].to(ref.F64), x["scale"]
    between = lambda i, j: torch.exp(g[i + 1:j + 1].sum())  # noqa: E731: from the write of i (-1: the start) to the read at j
    want = torch.zeros(5, dtype=ref.F64)
    last = 4
    for t in range(5):
        total = 0.0
        for i in range(t, 5):
            for j in range(-1, i):  # read at i of what is older than i
                w = S0 if j < 0 else k[j][:, None] * v[j][None]
                total += ((q[i][:, None] * w * dy[i][None] * s * between(j, i)) ** 2).sum()
            for j in range(i + 1, 6):  # written at i, read later, or left in the last state
                r = D0 if j > last else q[j][:, None] * dy[j][None] * s
                total += ((k[i][:, None] * v[i][None] * r * between(i, min(j, last))) ** 2).sum()
        for j in range(-1, 5):
            w = S0 if j < 0 else k[j][:, None] * v[j][None]
            total += ((w * D0 * between(j, last)) ** 2).sum()
        want[t] = total
    assert torch.allclose(bounds.spread(x)[0, :, 0], want, rtol=1e-10)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_cut_is_the_planned_one(dtype):
    if not os.path.exists(ssm.library_path()):
        pytest.skip("libssm.so not built")
    for backward in (False, True):
        seen = set()
        for b, H in ((1, 1), (1, 2), (1, 25), (1, 40), (2, 20), (1, 65), (1, 100), (3, 43), (1, 129), (4, 65)):
            for L in (1, 64, 255, 257, 600, 1100, 1600, 2500, 8191, 65536):
                segs, parts, _ = bounds.cut(b, L, H, dtype, backward)
                assert bounds.parts_of(b, L, H, dtype, backward) == (segs - 1) * parts, (b, H, L, backward)
                seen.add((segs > 1, parts > 1))
        assert seen == {(False, False), (True, False), (True, True)}
