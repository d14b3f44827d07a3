"""The norms around a block on the GPU, through the C ABI, against the definition in float64 and its gradients by the chain
rule of torch.

Bounds.  A value is a product and sum of a few floats, each off by 2^-24 of its magnitude at most, with sums over W
elements (rows) or over the rows (parameters) of 2^-24 a term, and is then rounded to its type (half a step, 2^-8 of a value
in bf16).  Magnitudes are those of the definition with every term counted positive: the square roots' and the norms'
mean terms are included, the silu's argument z adds |z| 2^-24 of it by the exponential.
"""
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu
EPS = 1e-5
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def make(rows=5, H=1, W=96, dtype="bf16", post=True, pre=True, gate=True, residual="same", scale=True, weights=True, seed=0):
    import torch

    gen = torch.Generator().manual_seed(seed)
    io = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    res = {"none": None, "same": io, "f32": torch.float32}[residual]
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    shape, par = ((rows, W), (W,)) if H == 1 else ((rows, H, W), (H, W))
    c = lambda t, d=torch.float32: t.to(d).cuda()  # noqa: E731
    x = {"x": c(1.5 * n(*shape), io), "z": c(2 * n(*shape), io) if gate else None,
         "residual": None if res is None else c(2 * n(*shape), res),
         "post_weight": c(1 + 0.3 * n(*par)) if post and weights else None,
         "pre_weight": c(1 + 0.3 * n(*par)) if pre and weights else None, "scale": c(0.5 + 0.2 * n(*par)) if scale else None,
         "norms": "both" if post and pre else "post" if post else "pre"}
    return x, {"dh": c(n(*shape), res or io), "dn": c(n(*shape), io) if pre else None}


def definition(x, eps=EPS):
    """(h, n, rstd_post, rstd_pre) of float64 tensors."""
    import torch

    v = x["x"]
    r1 = r2 = n = None
    if x["norms"] != "pre":
        r1 = (v.square().mean(-1) + eps).rsqrt()
        v = v * r1[..., None] * (1 if x["post_weight"] is None else x["post_weight"])
    if x["z"] is not None:
        v = v * x["z"] * torch.sigmoid(x["z"])
    if x["scale"] is not None:
        v = v * x["scale"]
    h = v if x["residual"] is None else v + x["residual"]
    if x["norms"] != "post":
        r2 = (h.square().mean(-1) + eps).rsqrt()
        n = h * r2[..., None] * (1 if x["pre_weight"] is None else x["pre_weight"])
    return h, n, r1, r2


def f64(t):
    import torch

    return t.detach().cpu().double() if isinstance(t, torch.Tensor) else t


def close(got, want, mag, half, terms, what):
    import torch

    tol = (mag * (terms + 40) * 2.0 ** -24 + want.abs() * half) * 1.01 + 1e-37
    d = (got.detach().cpu().double() - want).abs()
    assert not torch.isnan(d).any(), f"{what} has NaN"
    over = (d / tol).max().item() if d.numel() else 0.0
    print(f"[blocknorm] {what} at {over:.3f} of its bound", flush=True)
    assert over <= 1.0, f"{what} is {over:.3f} times its bound"


def check(x, d, what, param_grads=True):
    import torch

    import selective_state_space_35_amd as ssm

    say(what)
    names = ("post_weight", "z", "scale", "residual", "pre_weight", "norms")
    given = {k: x[k] for k in names}
    H = None if x["x"].dim() == 2 else x["x"].shape[1]
    h, n, r1, r2 = ssm.ssm_blocknorm_fwd(x["x"], **given, eps=EPS, heads=H)
    torch.cuda.synchronize()
    ref = {k: f64(t) for k, t in x.items()}
    leaves = {k: t.clone().requires_grad_() for k, t in ref.items() if isinstance(t, torch.Tensor)}
    wh, wn, w1, w2 = definition({**ref, **leaves})
    io = "f32" if x["x"].dtype == torch.float32 else "bf16"
    rio = "f32" if h.dtype == torch.float32 else "bf16"
    W = x["x"].shape[-1]
    zmag = 1 if ref["z"] is None else 1 + ref["z"].abs()
    part = (wh if ref["residual"] is None else wh - ref["residual"]).detach().abs() * zmag
    mag = part + (0 if ref["residual"] is None else ref["residual"].abs())
    # a row's rstd is off by half the relative error of its mean: W / 2 terms at most
    close(h, wh.detach(), mag * (1 if w1 is None else 1) + part * W / 40, HALF[rio], 0, what + " h")
    if w1 is not None:
        close(r1, w1.detach(), w1.detach(), 2.0 ** -24, W, what + " rstd_post")
    else:
        assert r1 is None
    if w2 is not None:
        close(r2, w2.detach(), w2.detach() * zmag.max() if ref["z"] is not None else w2.detach(), 2.0 ** -24, 2 * W, what + " rstd_pre")
        pw = 1 if ref["pre_weight"] is None else ref["pre_weight"].abs()
        close(n, wn.detach(), (mag + part * W / 40) * w2.detach()[..., None] * pw + wn.detach().abs() * W / 20, HALF[io], 0, what + " n")
    else:
        assert r2 is None and n is None
    loss = (wh * f64(d["dh"])).sum() + (0 if wn is None else (wn * f64(d["dn"])).sum())
    loss.backward()
    say(what + ", backward")
    got = ssm.ssm_blocknorm_bwd(x["x"], r1, r2, dh=d["dh"], dn=d["dn"], **given, heads=H, param_grads=param_grads)
    torch.cuda.synchronize()
    # magnitudes: the chain with every term positive
    with torch.no_grad():
        a = lambda t: 1.0 if t is None else t.abs()  # noqa: E731
        u = part / a(ref["scale"])
        e = f64(d["dh"]).abs()
        hh = None
        if w2 is not None:
            r = w2[..., None]
            hh = mag * r
            t = f64(d["dn"]).abs() * a(ref["pre_weight"])
            e = e + r * (t + hh * (t * hh).mean(-1, keepdim=True))
        c = e * a(ref["scale"])
        s = 1.0 if ref["z"] is None else (ref["z"] * torch.sigmoid(ref["z"])).abs() * zmag
        p = ref["x"].abs() * (1 if w1 is None else w1[..., None] * a(ref["post_weight"]))
        dd = c * s
        xh = None
        dx = dd
        if w1 is not None:
            xh = ref["x"].abs() * w1[..., None]
            dd = dd * a(ref["post_weight"])
            dx = w1[..., None] * (dd + xh * (dd * xh).mean(-1, keepdim=True))
        mags = {"x": dx, "residual": e, "z": c * p * (1 if ref["z"] is None else 2 * zmag)}
        R = x["x"].shape[0]
        mags["scale"] = (e * u).sum(0)
        if w1 is not None:
            mags["post_weight"] = (c * s * xh).sum(0)
        if w2 is not None:
            mags["pre_weight"] = (f64(d["dn"]).abs() * hh).sum(0)
    for k in ("x", "z", "residual", "post_weight", "scale", "pre_weight"):
        g = got["d" + k]
        if k not in leaves or (not param_grads and k in ("post_weight", "scale", "pre_weight")):
            assert g is None, k
            continue
        half = HALF["f32" if g.dtype == torch.float32 else "bf16"]
        terms = 4 * W + (R if g.dtype == torch.float32 and k in ("post_weight", "scale", "pre_weight") else 0)
        close(g, leaves[k].grad, mags[k], half, terms, what + " d" + k)


FORMS = [dict(post=True, pre=True, gate=False, residual="same"), dict(post=True, pre=True, gate=True, residual="f32"),
         dict(post=True, pre=False, gate=True, residual="none", scale=False), dict(post=False, pre=True, gate=False, residual="none", scale=False),
         dict(post=False, pre=True, gate=False, residual="same"), dict(post=True, pre=False, gate=False, residual="f32"),
         dict(post=False, pre=True, gate=True, residual="same", weights=False, scale=False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("H,W", [(1, 96), (3, 40), (1, 33), (5, 7)])
def test_forms(H, W, form, dtype):
    check(*make(rows=11, H=H, W=W, dtype=dtype, seed=form, **FORMS[form]), f"blocknorm form {form} H={H} W={W} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 2, 8, 63, 64, 65, 128, 129, 256, 257, 512, 513, 1000, 1001, 1536, 2047, 2048, 2049, 2560, 4096, 5120,
                               5121, 8192, 8193, 10240, 16383, 16384])
def test_widths(W, dtype):
    check(*make(rows=3, W=W, dtype=dtype, seed=W), f"blocknorm W={W} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H,W", [(1, 1, 1536), (2, 1, 2560), (700, 1, 320), (1, 40, 128), (130, 24, 64), (5000, 1, 24), (2100, 7, 16)])
def test_rows(rows, H, W, dtype):
    check(*make(rows=rows, H=H, W=W, dtype=dtype, seed=rows), f"blocknorm rows={rows} H={H} W={W} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(dtype):
    import torch

    import selective_state_space_35_amd as ssm

    x, d = make(rows=0, dtype=dtype)
    h, n, r1, r2 = ssm.ssm_blocknorm_fwd(**x)
    g = ssm.ssm_blocknorm_bwd(x["x"], r1, r2, **d, **{k: x[k] for k in x if k != "x"})
    torch.cuda.synchronize()
    assert h.shape == (0, 96) and n.shape == (0, 96) and r1.shape == (0,)
    for k in ("dpost_weight", "dscale", "dpre_weight"):
        assert (g[k] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_tensors_and_repeats(dtype):
    """Tensors that begin one element behind an aligned address, without the parameters' gradients, and twice."""
    import torch

    import selective_state_space_35_amd as ssm

    for form in (0, 1):
        x, d = make(rows=9, W=128, dtype=dtype, seed=4, **FORMS[form])
        for src in (x, d):
            for k, t in src.items():
                if isinstance(t, torch.Tensor):
                    room = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
                    room[1:] = t.reshape(-1)
                    src[k] = room[1:].view(t.shape)
        check(x, d, f"blocknorm unaligned {dtype}")
        check(x, d, f"blocknorm unaligned, no parameters {dtype}", param_grads=False)
    x, d = make(rows=300, W=256, dtype=dtype, seed=5)
    given = {k: x[k] for k in x if k != "x"}
    runs = []
    for _ in range(2):
        h, n, r1, r2 = ssm.ssm_blocknorm_fwd(x["x"], **given)
        runs.append((h, n, r1, r2, *ssm.ssm_blocknorm_bwd(x["x"], r1, r2, **d, **given).values()))
    _, n2, _, _ = ssm.ssm_blocknorm_fwd(x["x"], **given, return_h=False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*runs)) and torch.equal(n2, runs[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row(bad, dtype):
    import torch

    import selective_state_space_35_amd as ssm

    for W in (64, 320, 33):
        x, d = make(rows=12, W=W, dtype=dtype, seed=6)
        given = {k: x[k] for k in x if k != "x"}
        h0, n0, r1, r2 = ssm.ssm_blocknorm_fwd(x["x"], **given)
        g0 = ssm.ssm_blocknorm_bwd(x["x"], r1, r2, **d, **given)
        y = x["x"].clone()
        y[5, 7] = bad
        h, n, s1, s2 = ssm.ssm_blocknorm_fwd(y, **given)
        g = ssm.ssm_blocknorm_bwd(y, s1, s2, **d, **given)
        torch.cuda.synchronize()
        other = [i for i in range(12) if i != 5]
        for a, b in ((h, h0), (n, n0), (g["dx"], g0["dx"]), (g["dz"], g0["dz"]), (g["dresidual"], g0["dresidual"])):
            assert torch.equal(a[other], b[other])
        assert not torch.isfinite(n[5]).all()


def test_rows_of_zeros():
    import torch

    import selective_state_space_35_amd as ssm

    x = torch.zeros(3, 64, device="cuda")
    h, n, r1, r2 = ssm.ssm_blocknorm_fwd(x, norms="both", eps=1e-5)
    torch.cuda.synchronize()
    assert (h == 0).all() and (n == 0).all() and torch.allclose(r1, torch.full_like(r1, 1e-5 ** -0.5))


def test_keys_of_length_one():
    """The norm before a block alone, with 1 / sqrt(W): rows of length one."""
    import torch

    import selective_state_space_35_amd as ssm

    k = torch.randn(2, 50, 4, 32, device="cuda")
    w = torch.full((4, 32), 32 ** -0.5, device="cuda")
    h, n, _, _ = ssm.ssm_blocknorm_fwd(k, pre_weight=w, norms="pre", eps=0.0, return_h=False)
    torch.cuda.synchronize()
    assert h is None and torch.allclose(n.norm(dim=-1), torch.ones(2, 50, 4, device="cuda"), atol=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph(dtype):
    """Captured, and replayed with other inputs."""
    import torch

    import selective_state_space_35_amd as ssm

    x, d = make(rows=300, W=640, dtype=dtype, seed=7)
    given = {k: x[k] for k in x if k != "x"}

    def both():
        h, n, r1, r2 = ssm.ssm_blocknorm_fwd(x["x"], **given)
        return (h, n, r1, r2, *ssm.ssm_blocknorm_bwd(x["x"], r1, r2, **d, **given).values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (8, 9, 10):
        y, e = make(rows=300, W=640, dtype=dtype, seed=seed)
        for src, new in ((x, y), (d, e)):
            for k, t in src.items():
                if isinstance(t, torch.Tensor):
                    t.copy_(new[k])
        want = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [3, 7, 9, 12, 14, 77, 1029, 5115])
def test_rows_that_end_inside_a_piece(W, dtype):
    """Widths that are not whole 16-byte pieces, from any address: what lies around the tensors is not read into a result
    (it is NaN), and not written."""
    import torch

    import selective_state_space_35_amd as ssm

    for form in (0, 1, 2, 6):
        x, d = make(rows=5, W=W, dtype=dtype, seed=W + form, **FORMS[form])
        for off, src in ((3, x), (5, d)):
            for k, t in src.items():
                if isinstance(t, torch.Tensor):
                    room = torch.full((t.numel() + 16,), float("nan"), dtype=t.dtype, device="cuda")
                    room[off:off + t.numel()] = t.reshape(-1)
                    src[k] = room[off:off + t.numel()].view(t.shape)
        check(x, d, f"blocknorm piece W={W} form {form} {dtype}")
        given = {k: x[k] for k in x if k != "x"}
        h0, n0, _, _ = ssm.ssm_blocknorm_fwd(x["x"], **given)
        into = {}
        for k, t in (("h", h0), ("n", n0)):
            if t is not None:
                room = torch.full((t.numel() + 24,), 7.0, dtype=t.dtype, device="cuda")
                into[k] = (room, t, room[11:11 + t.numel()].view(t.shape))
        ssm.ssm_blocknorm_fwd(x["x"], **given, **{k: v[2] for k, v in into.items()})
        torch.cuda.synchronize()
        for k, (room, want, got) in into.items():
            assert torch.equal(got, want), k
            assert (room[:11] == 7).all() and (room[11 + want.numel():] == 7).all(), k
