"""The float64 reference of the gated delta rule: its gradients against torch's chain rule and differences, special cases in
closed form, and its bounds against a lost rounding (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from tests import deltarule_ref as ref  # noqa: E402


def make(b=2, L=20, H=4, G=2, Dk=6, Dv=5, seed=0, lengths=None):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, dtype=ref.F64)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    return {"q": unit(n(b, L, G, Dk)), "k": unit(n(b, L, G, Dk)), "v": n(b, L, H, Dv), "beta": torch.sigmoid(n(b, L, H)),
            "g": -0.2 * n(b, L, H).abs(), "A": -0.1 * n(H).abs(), "dy": n(b, L, H, Dv), "initial_state": n(b, H, Dk, Dv),
            "d_last_state": n(b, H, Dk, Dv), "scale": 0.4,
            "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}


def loss_of(x):
    """The recurrence once more, of the definition as it reads."""
    b, L, H, Dv = x["v"].shape
    G = x["q"].shape[2]
    total = 0.0
    for i in range(b):
        n = L if x["lengths"] is None else min(max(int(x["lengths"][i]), 0), L)
        for h in range(H):
            S = x["initial_state"][i, h]
            for t in range(n):
                k = x["k"][i, t, h // (H // G)]
                S = S * torch.exp(x["A"][h] + x["g"][i, t, h])
                S = S + torch.outer(k, x["beta"][i, t, h] * (x["v"][i, t, h] - S.T @ k))
                total = total + (x["scale"] * (S.T @ x["q"][i, t, h // (H // G)]) * x["dy"][i, t, h]).sum()
            total = total + (S * x["d_last_state"][i, h]).sum()
    return total


@pytest.mark.parametrize("lengths", [None, [7, 0]])
def test_gradients(lengths):
    x = make(lengths=lengths)
    names = ("q", "k", "v", "beta", "g", "initial_state")
    leaves = {n: x[n].clone().requires_grad_() for n in names}
    loss = loss_of(dict(x, **leaves))
    loss.backward()
    f, _ = ref.forward(x)
    assert torch.allclose((f["y"] * x["dy"]).sum() + (f["last_state"] * x["d_last_state"]).sum(), loss.detach(), rtol=1e-12)
    d, V = ref.backward(x)
    for n in names:
        got = d["d_initial_state" if n == "initial_state" else "d" + n]
        assert torch.allclose(got, leaves[n].grad, rtol=1e-10, atol=1e-12), n
        at = tuple(min(3, s - 1) for s in x[n].shape)
        vals = []
        for e in (1e-5, -1e-5):
            z = x[n].clone()
            z[at] += e
            vals.append(loss_of(dict(x, **{n: z})).item())
        assert abs((vals[0] - vals[1]) / 2e-5 - got[at].item()) < 1e-6, n
    assert all((t >= 0).all() for t in V.values())


def test_without_the_old_answer_it_is_linear_attention():
    """Keys orthogonal to all others: nothing is taken out, and the rule is linear attention with beta v."""
    from tests import linattn_ref

    x = make(L=6, Dk=6, H=2, G=2)
    x["k"] = torch.eye(6, dtype=ref.F64)[None, :, None].expand(2, 6, 2, 6).contiguous()
    x["initial_state"] = None
    f, _ = ref.forward(x)
    want = linattn_ref.forward(dict(x, v=x["beta"][..., None] * x["v"]))
    for n in ("y", "last_state"):
        assert torch.allclose(f[n], want[n], rtol=1e-12), n


def test_a_key_of_length_one_is_answered_with_its_value():
    x = make(H=2, G=2)
    x["beta"] = torch.ones_like(x["beta"])
    x["q"], x["scale"] = x["k"], 1.0
    f, _ = ref.forward(x)
    assert torch.allclose(f["y"], x["v"], rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bounds_refuse_one_lost_rounding(dtype):
    """The recurrence in the type's own arithmetic is within the bounds; with what a token writes rounded once to bf16 (in a
    float call, to 16 bits) it is not."""
    x = make(b=1, L=120, Dk=32, Dv=32, H=2, G=2, seed=3)
    x = {k: t.to(dtype if k in ("q", "k", "v", "beta", "g", "dy") else torch.float32) if isinstance(t, torch.Tensor) else t for k, t in x.items()}
    want, V = ref.forward(x)

    def run(rough):
        q, k, v, beta, r, _, S, scale = (t.to(torch.float32) if isinstance(t, torch.Tensor) else t for t in ref.inputs(x))
        y = torch.zeros_like(v)
        for t in range(v.shape[1]):
            S = S * r[:, t, :, None, None]
            u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(-2))
            u = u.to(torch.bfloat16).float() if rough == "bf16" else (u * 2.0 ** 10).to(torch.float16).float() * 2.0 ** -10 if rough else u
            S = S + k[:, t, :, :, None] * u[:, :, None, :]
            y[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
        return {"y": y.to(dtype), "last_state": S}

    for n, t in run("").items():
        ref.within(t, want[n], V[n], n, x, "plain")
    rough = run("bf16" if dtype == torch.bfloat16 else "f16")
    with pytest.raises(AssertionError, match="times its bound"):
        ref.within(rough["last_state"], want["last_state"], V["last_state"], "last_state", x, "rough")
