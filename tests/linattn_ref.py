"""Linear attention with a decay for each head in float64: the recurrence token by token, its
gradients by the chain rule, and bounds on what rounded arithmetic may add.

A bound is a magnitude times a rounding.  The magnitudes are the same recurrences on absolute values
(every product counted positive).  The roundings, with half a step of bf16 2^-8 and of fp32 2^-24:

* y, dq, dk, dv: the mixing matrix and the state are rounded once to the products' operand type
  (bf16: 2^-8 of the magnitude), sums run in fp32 over at most L + Dk + Dv + 64 terms, a decay is
  exp of an fp32 number (its argument's rounding is within the same count for |log decay| <= 64 a
  chunk), and the result is rounded to the output type (2^-8 of the value, fp32 none).
* states in float: the written products are split in two bf16 parts (2^-16 of the magnitude), the
  rest as above.
* dg: sums of fp32 products over the tokens after, each with the error of dq and dk before their
  rounding (two bf16 parts again), then rounded to the output type.
"""
import torch

F64 = torch.float64
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def heads(t, H):
    """[b, L, G, D] -> [b, L, H, D] float64 on the CPU."""
    return t.detach().cpu().to(F64).repeat_interleave(H // t.shape[2], dim=2)


def _inputs(x):
    v = x["v"].detach().cpu().to(F64)
    b, L, H, _ = v.shape
    lg = torch.zeros((b, L, H), dtype=F64)
    if x.get("A") is not None:
        lg = lg + x["A"].detach().cpu().to(F64)
    if x.get("g") is not None:
        lg = lg + x["g"].detach().cpu().to(F64)
    n = torch.full((b,), L) if x.get("lengths") is None else x["lengths"].cpu().long().clamp(0, L)
    live = torch.arange(L)[None] < n[:, None]
    r = torch.where(live[..., None], lg.exp(), torch.ones_like(lg))
    cut = lambda t: torch.where(live[..., None, None], t, torch.zeros_like(t))  # noqa: E731
    f = lambda t: None if t is None else t.detach().cpu().to(F64)  # noqa: E731
    return cut(heads(x["q"], H)), cut(heads(x["k"], H)), cut(v), r, live, cut, f


def forward(x, absolute=False):
    """{y, last_state}; with ``absolute`` of the inputs' absolute values."""
    q, k, v, r, live, cut, f = _inputs(x)
    a = (lambda t: t.abs()) if absolute else (lambda t: t)
    b, L, H, Dk = q.shape
    S = f(x.get("initial_state"))
    S = torch.zeros((b, H, Dk, v.shape[3]), dtype=F64) if S is None else a(S)
    y = torch.zeros_like(v)
    for t in range(L):
        S = S * r[:, t, :, None, None] + a(k[:, t])[..., None] * a(v[:, t])[..., None, :]
        y[:, t] = (a(q[:, t])[..., None] * S).sum(-2) * (abs(x["scale"]) if absolute else x["scale"])
    return {"y": cut(y), "last_state": S}


def backward(x, absolute=False):
    """{dq, dk, dv, dg, d_initial_state}; with ``absolute`` the magnitudes (dg's: of the suffix sums it is computed by)."""
    q, k, v, r, live, cut, f = _inputs(x)
    a = (lambda t: t.abs()) if absolute else (lambda t: t)
    q, k, v, dy = a(q), a(k), a(v), a(cut(f(x["dy"])))
    scale = abs(x["scale"]) if absolute else x["scale"]
    b, L, H, Dk = q.shape
    G = x["q"].shape[2]
    zero = torch.zeros((b, H, Dk, v.shape[3]), dtype=F64)
    S = zero if x.get("initial_state") is None else a(f(x["initial_state"]))
    D = zero if x.get("d_last_state") is None else a(f(x["d_last_state"]))
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(v), torch.zeros((b, L, H), dtype=F64)
    before = []
    read = torch.zeros((b, L, H), dtype=F64)
    for t in range(L):
        S = S * r[:, t, :, None, None]
        before.append(S)
        read[:, t] = (q[:, t] * (S * dy[:, t][..., None, :]).sum(-1)).sum(-1) * scale
        S = S + k[:, t][..., None] * v[:, t][..., None, :]
        dq[:, t] = (S * dy[:, t][..., None, :]).sum(-1) * scale
    tail = (D * S).sum((-1, -2))
    for t in range(L - 1, -1, -1):
        tail = tail + read[:, t] + (k[:, t] * (D * v[:, t][..., None, :]).sum(-1)).sum(-1)
        D = D + q[:, t][..., None] * dy[:, t][..., None, :] * scale
        dk[:, t] = (D * v[:, t][..., None, :]).sum(-1)
        dv[:, t] = (D * k[:, t][..., None]).sum(-2)
        dg[:, t] = tail if absolute else (D * before[t]).sum((-1, -2))
        D = D * r[:, t, :, None, None]
    group = lambda t: t.reshape(b, L, G, H // G, Dk).sum(3)  # noqa: E731
    return {"dq": group(cut(dq)), "dk": group(cut(dk)), "dv": cut(dv), "dg": dg * live[..., None], "d_initial_state": D}


def terms(x):
    b, L, H, Dv = x["v"].shape
    return L + x["q"].shape[3] + Dv + 64


def within(got, ref, mag, name, x, what):
    """Asserts the documented bound of output ``name`` elementwise."""
    io = x["v"].dtype
    fp = terms(x) * 2.0 ** -24
    if name in ("last_state", "d_initial_state"):
        tol = mag * ((2.0 ** -16 if io == torch.bfloat16 else 0.0) + 2 * fp)
    elif io == torch.bfloat16:
        part = 2.0 ** -16 if name == "dg" else 2.0 ** -8
        tol = mag * (part + 2 * fp) + ref.abs() * 2.0 ** -8
    else:
        tol = mag * 2 * fp + ref.abs() * 2.0 ** -24
    tol = tol * 1.01 + 1e-37
    d = (got.detach().cpu().to(F64) - ref).abs()
    assert not torch.isnan(d).any(), f"{what}: {name} has NaN"
    over = (d / tol).max().item() if d.numel() else 0.0
    print(f"[linattn] {what}: {name} at {over:.3f} of its bound, largest error {d.max().item() if d.numel() else 0:.2e}", flush=True)
    assert over <= 1.0, f"{what}: {name} is {over:.3f} times its bound"
