"""A mixer as a model uses it: norms of q and k per head, the gated delta rule, the gated norm of each head's outputs, the
residual and the norm before the next block, forward and backward, and then tokens on its states."""
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu


def inputs(dtype, b=2, L=150, H=4, G=2, D=48, seed=0):
    import torch

    gen = torch.Generator().manual_seed(seed)
    io = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    W = H * D
    x = {"q": n(b, L, G, D), "k": n(b, L, G, D), "v": n(b, L, H, D), "z": n(b, L, H, D), "beta": torch.sigmoid(n(b, L, H)),
         "g": -0.1 * n(b, L, H).abs()}
    x = {k: t.to(io).cuda() for k, t in x.items()}
    x["residual"] = n(b, L, W).cuda()  # the stream in float
    x["head_weight"] = (1 + 0.2 * n(H, D)).cuda()
    x["scale"] = (0.5 + 0.1 * n(W)).cuda()
    x["pre_weight"] = (1 + 0.2 * n(W)).cuda()
    x["dh"], x["dn"] = n(b, L, W).cuda(), n(b, L, W).to(io).cuda()
    x["unit"] = torch.full((G, D), D ** -0.5).cuda()
    return x


def definition(x, dtype=None):
    """(h, n, last) in the tensors' own type, from leaves."""
    import torch

    unit = lambda t: t * (t.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * t.shape[-1] ** -0.5  # noqa: E731
    b, L, H, D = x["v"].shape
    rep = H // x["q"].shape[2]
    q, k = (unit(x[n]).repeat_interleave(rep, dim=2) for n in ("q", "k"))
    S = torch.zeros((b, H, D, D), dtype=x["v"].dtype)
    ys = []
    for t in range(L):
        S = S * x["g"][:, t, :, None, None].exp()
        u = x["beta"][:, t, :, None] * (x["v"][:, t] - (k[:, t, :, :, None] * S).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        ys.append((q[:, t, :, :, None] * S).sum(-2) * D ** -0.5)
    y = torch.stack(ys, 1)
    o = y * (y.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * x["head_weight"] * torch.nn.functional.silu(x["z"])
    h = x["residual"] + x["scale"] * o.reshape(b, L, H * D)
    n = h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * x["pre_weight"]
    return h, n, S


def mixer(x):
    import torch

    import selective_state_space_35_amd as ssm

    b, L, H, D = x["v"].shape
    flat = (b, L, H * D)
    _, q, _, rq = ssm.ssm_blocknorm_fwd(x["q"], pre_weight=x["unit"], norms="pre", return_h=False)
    _, k, _, rk = ssm.ssm_blocknorm_fwd(x["k"], pre_weight=x["unit"], norms="pre", return_h=False)
    y, last = ssm.ssm_deltarule_fwd(q, k, x["v"], beta=x["beta"], g=x["g"])
    o, _, ro, _ = ssm.ssm_blocknorm_fwd(y, post_weight=x["head_weight"], z=x["z"], norms="post")
    h, n, _, rn = ssm.ssm_blocknorm_fwd(o.view(flat), scale=x["scale"], residual=x["residual"], pre_weight=x["pre_weight"], norms="pre")
    d = ssm.ssm_blocknorm_bwd(o.view(flat), None, rn, dh=x["dh"], dn=x["dn"], scale=x["scale"], residual=x["residual"],
                              pre_weight=x["pre_weight"], norms="pre")
    e = ssm.ssm_blocknorm_bwd(y, ro, dh=d["dx"].view(y.shape), post_weight=x["head_weight"], z=x["z"], norms="post")
    f = ssm.ssm_deltarule_bwd(q, k, x["v"], e["dx"], beta=x["beta"], g=x["g"])
    dq, dk = (ssm.ssm_blocknorm_bwd(x[name], None, r, dn=f["d" + name], pre_weight=x["unit"], norms="pre", param_grads=False)["dx"]
              for name, r in (("q", rq), ("k", rk)))
    grads = {"q": dq, "k": dk, "v": f["dv"], "beta": f["dbeta"], "g": f["dg"], "z": e["dz"], "head_weight": e["dpost_weight"],
             "scale": d["dscale"], "pre_weight": d["dpre_weight"], "residual": d["dresidual"]}
    return h, n, last, grads


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_mixer_with_its_norms(dtype):
    """In the norm of each output: a bf16 run rounds eight tensors in a row, each off by at most 2^-8 of its values and
    by 0.41 of that in the norm; a float one computes each with some hundred roundings of 2^-24."""
    import torch

    x = inputs(dtype)
    say(f"mixer {dtype}")
    h, n, last, grads = mixer(x)
    torch.cuda.synchronize()
    leaves = {k: x[k].cpu().double().requires_grad_() for k in grads}
    wh, wn, ws = definition(leaves)
    ((wh * x["dh"].cpu().double()).sum() + (wn * x["dn"].cpu().double()).sum()).backward()
    tol = 8 * 0.5 * 2.0 ** -8 if dtype == "bf16" else 300 * 2.0 ** -24
    for name, got, want in [("h", h, wh), ("n", n, wn), ("last", last, ws)] + [("d" + k, grads[k], leaves[k].grad) for k in grads]:
        rel = ((got.cpu().double() - want).norm() / want.norm()).item()
        print(f"[mixer] {name} {rel:.2e} (bound {tol:.1e})", flush=True)
        assert rel <= tol, (name, rel)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_tokens(dtype):
    """The states of a prompt carried on token by token are those of the whole sequence."""
    import torch

    import selective_state_space_35_amd as ssm

    x = inputs(dtype, L=140, seed=3)
    _, q, _, _ = ssm.ssm_blocknorm_fwd(x["q"], pre_weight=x["unit"], norms="pre", return_h=False)
    _, k, _, _ = ssm.ssm_blocknorm_fwd(x["k"], pre_weight=x["unit"], norms="pre", return_h=False)
    y, last = ssm.ssm_deltarule_fwd(q, k, x["v"], beta=x["beta"], g=x["g"])
    cut = lambda t, a, e: t[:, a:e].contiguous()  # noqa: E731
    yp, state = ssm.ssm_deltarule_fwd(*(cut(t, 0, 133) for t in (q, k, x["v"])), beta=cut(x["beta"], 0, 133), g=cut(x["g"], 0, 133))
    ys = [yp]
    for t in range(133, 140):
        q1, k1, v1, b1, g1 = (a[:, t].contiguous() for a in (q, k, x["v"], x["beta"], x["g"]))
        ys.append(ssm.ssm_deltarule_update(state, q1, k1, v1, beta=b1, g=g1)[:, None])
    torch.cuda.synchronize()
    tol = 2.0 ** -8 if dtype == "bf16" else 300 * 2.0 ** -24
    assert ((torch.cat(ys, 1).double() - y.double()).norm() / y.double().norm()).item() <= tol
    assert ((state.double() - last.double()).norm() / last.double().norm()).item() <= 300 * 2.0 ** -24


def test_streams_and_devices():
    """On a stream that is not the tensors' own, with the library's own workspace, and two calls on two streams at once."""
    import ctypes

    import torch

    import selective_state_space_35_amd as ssm

    x = inputs("bf16", L=300, seed=5)
    want = ssm.ssm_deltarule_fwd(x["q"] * 0.1, x["k"] * 0.1, x["v"], beta=x["beta"], g=x["g"])
    torch.cuda.synchronize()
    q, k = (x["q"] * 0.1).contiguous(), (x["k"] * 0.1).contiguous()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                outs.append(ssm.ssm_deltarule_fwd(q, k, x["v"], beta=x["beta"], g=x["g"]))
    torch.cuda.synchronize()
    for y, last in outs:
        assert torch.equal(y, want[0]) and torch.equal(last, want[1])
    lib = ssm.load_library()
    b, L, H, D = x["v"].shape
    y, last = torch.empty_like(want[0]), torch.empty_like(want[1])
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = lib.ssm_deltarule_fwd(p(q), p(k), p(x["v"]), p(x["beta"]), p(x["g"]), None, None, D ** -0.5, None, p(y), p(last), b, L,
                               H, q.shape[2], D, D, 1, None, 0, ctypes.c_void_p(streams[0].cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(last, want[1])
