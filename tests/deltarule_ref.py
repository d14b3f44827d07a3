"""The gated delta rule in float64: the recurrence token by token, its gradients by the chain rule, and how much rounded
arithmetic may add.

With keys of length one, 0 <= beta <= 2 and log decays of at most zero, a token's map of the state, r (I - beta k k^T), makes
no vector longer, and neither does its transpose, the map of the gradient.  So an error that a token's products put into a
column of the state never grows: its square adds to those before, of independent signs.  For column j of the state,

    E_j = r^2 E_j + beta^2 (v_j^2 + r^2 |S_j|^2)         (the squares of what a token's write is made of)

times the square of a unit is the expected square of the whole column's error, and so for D, the gradient of the state,
F_j = r^2 F_j + scale^2 |q|^2 dy_j^2 + beta^2 r^2 |D_j|^2.  An output's V adds to the squares of its own products those of its
operands' errors: y = scale S^T q has scale^2 (sum_i q_i^2 S_ij^2 + |q|^2 E_j), and so on.  The unit has two sides:

* float sums of ``terms`` products of random signs, 2^-24 sqrt(terms) (a state, in any type, and all outputs of float tensors);
* bf16 outputs: the operands of a product that are not given in bf16 are taken in two parts, each off by 2^-17 at most, in at
  most four products one after the other: 4 2^-16 with both operands so.

A value is held to eight times unit sqrt(V) (independent errors, fewer than 10^7 values a test) and half a step of its
own rounding: 2^-8 of it in bf16, 2^-24 in float.
"""
import torch

F64 = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SIGMAS = 8
CHUNK = 64  # the gate's gradient is a difference of sums over at most so many tokens


def _f(t):
    return None if t is None else t.detach().cpu().to(F64)


def inputs(x):
    """(q, k, v, beta, r, live, init, scale) in float64: q and k for every head, beta 0 and r 1 behind the lengths."""
    v = _f(x["v"])
    b, L, H, _ = v.shape
    q, k = (_f(x[n]).repeat_interleave(H // x[n].shape[2], dim=2) for n in ("q", "k"))
    lg = torch.zeros((b, L, H), dtype=F64)
    if x.get("A") is not None:
        lg = lg + _f(x["A"])
    if x.get("g") is not None:
        lg = lg + _f(x["g"])
    beta = torch.ones((b, L, H), dtype=F64) if x.get("beta") is None else _f(x["beta"])
    n = torch.full((b,), L) if x.get("lengths") is None else x["lengths"].cpu().long().clamp(0, L)
    live = torch.arange(L)[None] < n[:, None]
    cut = lambda t, at: torch.where(live.reshape(b, L, *[1] * (t.dim() - 2)), t, torch.full_like(t, at))  # noqa: E731
    init = _f(x.get("initial_state"))
    if init is None:
        init = torch.zeros((b, H, k.shape[3], v.shape[3]), dtype=F64)
    return cut(q, 0.0), cut(k, 0.0), cut(v, 0.0), cut(beta, 0.0), cut(lg.exp(), 1.0), live, init, x["scale"]


def forward(x):
    """({y, last_state}, their V)."""
    q, k, v, beta, r, live, S, scale = inputs(x)
    E = torch.zeros_like(v[:, 0])
    y, V = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(v.shape[1]):
        S, E, _, _, _ = _step(S, E, k[:, t], v[:, t], beta[:, t], r[:, t])
        y[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
        V[:, t] = scale ** 2 * ((q[:, t, :, :, None] * S).square().sum(-2) + q[:, t].square().sum(-1, keepdim=True) * E)
    alive = live[:, :, None, None]
    return {"y": y * alive, "last_state": S}, {"y": V * alive, "last_state": (S.square() + E[:, :, None, :])}


def _step(S, E, k, v, beta, r):
    r = r[..., None]
    P = S * r[..., None]
    E = E * r ** 2 + beta[..., None] ** 2 * (v.square() + P.square().sum(-2))
    left = v - (k[..., None] * P).sum(-2)
    u = beta[..., None] * left
    return P + k[..., None] * u[..., None, :], E, P, left, u


def backward(x):
    """({dq, dk, dv, dbeta, dg, d_initial_state}, their V)."""
    q, k, v, beta, r, live, S, scale = inputs(x)
    b, L, H, Dv = v.shape
    G, Dk = x["q"].shape[2:]
    dy = torch.where(live[:, :, None, None], _f(x["dy"]), torch.zeros_like(v))
    D = _f(x.get("d_last_state"))
    D = torch.zeros((b, H, Dk, Dv), dtype=F64) if D is None else D
    E, F = torch.zeros_like(v[:, 0]), torch.zeros_like(v[:, 0])
    kept = []
    for t in range(L):
        S, E2, P, left, u = _step(S, E, k[:, t], v[:, t], beta[:, t], r[:, t])
        kept.append((P, left, u, S, E, E2))
        E = E2
    z = lambda *s: torch.zeros(s, dtype=F64)  # noqa: E731
    d = {"dq": z(b, L, H, Dk), "dk": z(b, L, H, Dk), "dv": torch.zeros_like(v), "dbeta": z(b, L, H), "dg": z(b, L, H)}
    V = {n: torch.zeros_like(t) for n, t in d.items()}
    own = z(b, L, H)
    col = lambda t: t[..., None, :]  # noqa: E731
    for t in range(L - 1, -1, -1):
        P, left, u, S, E, E2 = kept[t]
        kt, qt, gt = k[:, t], q[:, t], dy[:, t]
        bt, rt = beta[:, t][..., None], r[:, t][..., None]
        d["dq"][:, t] = scale * (S * col(gt)).sum(-1)
        V["dq"][:, t] = scale ** 2 * ((S * col(gt)).square().sum(-1) + (E2 * gt ** 2).sum(-1, keepdim=True))
        D = D + scale * qt[..., None] * col(gt)
        F = F + scale ** 2 * qt.square().sum(-1, keepdim=True) * gt ** 2
        du = (kt[..., None] * D).sum(-2)
        dl = bt * du
        d["dv"][:, t] = dl
        V["dv"][:, t] = bt ** 2 * ((kt[..., None] * D).square().sum(-2) + F)
        d["dbeta"][:, t] = (du * left).sum(-1)
        V["dbeta"][:, t] = ((du * left).square() + (D.square().sum(-2) + F) * left ** 2 + du ** 2 * (v[:, t] ** 2 + P.square().sum(-2) + E)).sum(-1)
        d["dk"][:, t] = (D * col(u)).sum(-1) - (P * col(dl)).sum(-1)
        V["dk"][:, t] = ((D * col(u)).square() + (P * col(dl)).square()).sum(-1) + (
            F * u ** 2 + D.square().sum(-2) * bt ** 2 * E + E * dl ** 2 + P.square().sum(-2) * bt ** 2 * F).sum(-1, keepdim=True)
        own[:, t] = (scale ** 2 * (qt[..., None] * S * col(gt)).square() + (kt[..., None] * D * col(u)).square()
                     + (kt[..., None] * P * col(dl)).square()).sum((-1, -2))
        F = F + bt ** 2 * D.square().sum(-2)
        D = D - kt[..., None] * col(dl)
        d["dg"][:, t] = (D * P).sum((-1, -2))
        V["dg"][:, t] = (D * P).square().sum((-1, -2)) + (F * P.square().sum(-2) + E * D.square().sum(-2)).sum(-1)
        D = D * rt[..., None]
        F = F * rt ** 2
    for c in range(0, L, CHUNK):
        V["dg"][:, c:c + CHUNK] += own[:, c:c + CHUNK].sum(1, keepdim=True)
    for name in ("dq", "dk"):
        d[name] = d[name].reshape(b, L, G, H // G, Dk).sum(3)
        V[name] = V[name].reshape(b, L, G, H // G, Dk).sum(3)
    for name, t in d.items():
        alive = live.reshape(b, L, *[1] * (t.dim() - 2))
        d[name], V[name] = t * alive, V[name] * alive
    d["d_initial_state"], V["d_initial_state"] = D, D.square() + F[:, :, None, :]
    return d, V


def terms(x):
    b, L, H, Dv = x["v"].shape
    return L + x["q"].shape[3] + Dv + 64


def within(got, ref, V, name, x, what):
    """Asserts the documented bound of output ``name`` value by value."""
    io = x["v"].dtype
    unit = 2.0 ** -24 * terms(x) ** 0.5
    half = HALF[torch.float32]
    if name not in ("last_state", "d_initial_state"):
        half = HALF[io]
        if io == torch.bfloat16:
            unit += 4 * 2.0 ** -16
    tol = SIGMAS * unit * V.sqrt() + half * ref.abs() * 1.01 + 1e-30
    d = (got.detach().cpu().to(F64) - ref).abs()
    assert not torch.isnan(d).any(), f"{what}: {name} has NaN"
    over = (d / tol).max().item() if d.numel() else 0.0
    print(f"[deltarule] {what}: {name} at {over:.3f} of its bound, largest error {d.max().item() if d.numel() else 0:.2e}", flush=True)
    assert over <= 1.0, f"{what}: {name} is {over:.3f} times its bound"
