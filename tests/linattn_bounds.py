"""Bounds of linear attention's gate gradients and of its states that one lost rounding breaks, and how a call's
sequence is cut.

dg_t is a sum of products over the tokens from t on, each with a rounding error of its own sign, so its error grows as the
root of the sum of their squares, V_t: the gradient's recurrences on squared inputs, every term positive.  In units of
sqrt(V_t):

* bf16: the operands of a product are taken in two parts, off by 2^-16 of it at most, four times (the mixing
  weights or the state, written and read, in both dots).  Taken in one part they would be off by 2^-8, of which the
  root mean square is 0.4: 25 times as much.
* both: float sums of ``terms`` products of random signs, 2^-24 sqrt(terms).

Then the rounding of dg itself: half a step at most, as a root mean square over many values 1 / sqrt(3) of that where all of
them begin at a power of two, and 0.7 with a margin of three of its standard deviations over 64 values.
"""
import torch

from tests import linattn_ref as ref


def squares(x):
    """The inputs whose recurrences have the squares of those of x as their products."""
    z = dict(x)
    for k in ("q", "k", "v", "dy", "initial_state", "d_last_state"):
        if z.get(k) is not None:
            z[k] = z[k].detach().cpu().to(ref.F64) ** 2
    for k in ("g", "A"):
        if z.get(k) is not None:
            z[k] = z[k].detach().cpu().to(ref.F64) * 2
    z["scale"] = x["scale"] ** 2
    return z


def spread(x):
    """V [b, L, H]."""
    return ref.backward(squares(x), absolute=True)["dg"]


def dg_over(got, want, V, x, window=64):
    """The largest ratio of dg's root-mean-square error to its bound, over each head's tokens and over windows of them."""
    io = x["v"].dtype
    unit = 2.0 ** -24 * ref.terms(x) ** 0.5 + (4 * 2.0 ** -16 if io == torch.bfloat16 else 0.0)
    err2 = (got.detach().cpu().to(ref.F64) - want).square()
    tol2 = (unit ** 2) * V + (0.7 * ref.STEP[io] * want) ** 2
    worst = 0.0
    L = want.shape[1]
    for w in {min(window, L), L}:
        for t in range(0, L - w + 1, max(1, w // 2)):
            e, m = err2[:, t:t + w].mean(1), tol2[:, t:t + w].mean(1)
            worst = max(worst, (e / (m + 1e-60)).sqrt().max().item())
    return worst


def state_over(got, want, x, name):
    """The ratio of the error of ``last_state`` or ``d_initial_state`` to its bound, root mean squares: float sums of products
    of random signs, 2^-24 sqrt(terms) of the root of their squares, and nothing of a product lost before (two bf16 parts
    of what is written would be off by 0.4^2 2^-16, which is more up to 1500 tokens)."""
    f = ref.forward if name == "last_state" else ref.backward
    spread2 = f(squares(x), absolute=True)[name]
    e = (got.detach().cpu().to(ref.F64) - want).square().mean().sqrt()
    return (e / (spread2.mean().sqrt() * 2.0 ** -24 * ref.terms(x) ** 0.5)).item()


def cut(b, L, H, dtype, backward):
    """(segments, parts of all but the last, chunks a part) of a call, as the library plans it: segments for 256 workgroups,
    of at least 4 chunks, their states in parts for 512."""
    chunk = 64 if dtype == "bf16" else 32
    n = -(-L // chunk)
    heads = b * H
    want = max(1, 256 // (heads * (3 if backward else 1)))
    segs = min(want, max(1, n // 4))
    seg = max(1, -(-n // segs))
    parts = 1
    if segs > 1:
        parts = max(1, min(512 // (heads * (segs - 1) * (2 if backward else 1)), seg // 4))
    per = -(-seg // parts)
    segs = max(1, -(-n // (per * parts)))
    return segs, parts, per


def parts_of(b, L, H, dtype, backward):
    """The states a call keeps for each head of a batch row, from the workspace it asks for (of which nothing else grows
    with Dv)."""
    import selective_state_space_35_amd as ssm

    wide, narrow = (ssm.ssm_linattn_workspace(b, L, H, H, 64, Dv, dtype, backward) for Dv in (128, 64))
    return (wide - narrow) // (64 * 64 * 4 * b * H * (2 if backward else 1))
