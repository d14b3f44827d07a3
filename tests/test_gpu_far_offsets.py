"""The gated delta rule and the norms around a block where tensors have more than 2^31 elements: what lies at the far end is, bit
for bit, what the same data gives at the near end."""
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory_goes_back():
    yield
    import torch

    torch.cuda.empty_cache()


def randn(*shape, dtype=None, std=1.0, seed=0):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype or torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - a)
        flat[a:a + n] = (torch.randn(n, generator=gen, device="cuda") * std).to(out.dtype)
    return out


def test_batch_rows():
    """33 rows of 16384 tokens, 32 heads of 128: the last row lies behind 2^31 elements."""
    import torch

    import selective_state_space_35_amd as ssm

    b, L, H, D = 33, 16384, 32, 128
    assert (b - 1) * L * H * D >= 2 ** 31
    x = {k: randn(b, L, H, D, std=D ** -0.5 if k in "qk" else 1.0, seed=i) for i, k in enumerate(("q", "k", "v", "dy"))}
    x["k"] *= 0.9
    x["beta"], x["g"] = torch.sigmoid(randn(b, L, H, seed=5)), -0.1 * randn(b, L, H, seed=6).abs()
    for t in x.values():
        t[b - 1] = t[0]
    say("deltarule far batch row")
    y, last = ssm.ssm_deltarule_fwd(x["q"], x["k"], x["v"], beta=x["beta"], g=x["g"])
    d = ssm.ssm_deltarule_bwd(x["q"], x["k"], x["v"], x["dy"], beta=x["beta"], g=x["g"])
    torch.cuda.synchronize()
    assert torch.isfinite(last).all() and (y[0] != 0).any()
    assert torch.equal(y[0], y[b - 1]) and torch.equal(last[0], last[b - 1]) and not torch.equal(y[0], y[1])
    for k in ("dq", "dk", "dv", "dbeta", "dg"):
        assert torch.equal(d[k][0], d[k][b - 1]), k


def test_one_long_row():
    """One row of 524416 tokens: its last two chunks are the first two again, behind a reset."""
    import torch

    import selective_state_space_35_amd as ssm

    L, H, D, n = 524288 + 128, 32, 128, 128
    assert (L - n) * H * D >= 2 ** 31
    x = {k: randn(1, L, H, D, std=D ** -0.5 if k in "qk" else 1.0, seed=i) for i, k in enumerate(("q", "k", "v", "dy"))}
    x["k"] *= 0.9
    x["beta"], x["g"] = torch.sigmoid(randn(1, L, H, seed=5)), -0.1 * randn(1, L, H, seed=6).abs()
    x["g"][:, 0] = float("-inf")
    x["g"][:, n] = float("-inf")  # what follows the first two chunks does not come into their gradients either
    for t in x.values():
        t[:, L - n:] = t[:, :n]
    say("deltarule far tokens")
    y, last = ssm.ssm_deltarule_fwd(x["q"], x["k"], x["v"], beta=x["beta"], g=x["g"])
    d = ssm.ssm_deltarule_bwd(x["q"], x["k"], x["v"], x["dy"], beta=x["beta"], g=x["g"])
    torch.cuda.synchronize()
    assert torch.isfinite(last).all() and (y != 0).any()
    assert torch.equal(y[:, :n], y[:, L - n:])
    for k in ("dq", "dk", "dv", "dbeta", "dg"):
        assert torch.equal(d[k][:, :n], d[k][:, L - n:]), k


def test_states_of_a_token_step():
    import torch

    import selective_state_space_35_amd as ssm

    b, H, D = 1025, 128, 128
    assert (b - 1) * H * D * D >= 2 ** 31
    state = randn(b, H, D, D, dtype=torch.float32)
    state[b - 1] = state[0]
    q, k, v = (randn(b, H, D, std=D ** -0.5 if s < 2 else 1.0, seed=s) for s in range(3))
    beta = torch.sigmoid(randn(b, H, seed=4))
    for t in (q, k, v, beta):
        t[b - 1] = t[0]
    say("deltarule far states")
    y = ssm.ssm_deltarule_update(state, q, k, v, beta=beta)
    torch.cuda.synchronize()
    assert torch.equal(state[0], state[b - 1]) and torch.equal(y[0], y[b - 1]) and not torch.equal(y[0], y[1])


@pytest.mark.parametrize("norms,W", [("both", 1280), ("pre", 1281), ("post", 64)])
def test_rows_of_the_norms(norms, W):
    import torch

    import selective_state_space_35_amd as ssm

    rows = 2 ** 31 // W + 600
    x, r = randn(rows, W, seed=1), randn(rows, W, seed=2)
    z = randn(rows, W, seed=3) if norms == "post" else None
    dh, dn = randn(rows, W, seed=4), randn(rows, W, seed=5) if norms != "post" else None
    for t in (x, r, z, dh, dn):
        if t is not None:
            t[-500:] = t[:500]
    kw = dict(residual=r, z=z, norms=norms)
    say(f"blocknorm far rows W={W} {norms}")
    h, n, r1, r2 = ssm.ssm_blocknorm_fwd(x, **kw)
    d = ssm.ssm_blocknorm_bwd(x, r1, r2, dh=dh, dn=dn, **kw)
    torch.cuda.synchronize()
    for k, t in (("h", h), ("n", n), ("rstd_post", r1), ("rstd_pre", r2), ("dx", d["dx"]), ("dz", d["dz"]), ("dresidual", d["dresidual"])):
        assert t is None or torch.equal(t[:500], t[-500:]), k
    assert torch.isfinite(h[-500:]).all() and (h[-500:] != 0).any()
