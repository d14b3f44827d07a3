"""Layer norm on the GPU, through the C ABI, against float64.

Bounds, with u = 2^-24 (half a step of fp32) and o half a step of the output type (2^-8 or 2^-24):
* mean: W / 2 + 8 roundings of sums of |x|: (W + 16) u mean|x|, far above what trees of sums give.
* rstd: the centred squares are sums of non-negative values: relative (W + 32) u, and half of it
  passes through the root; a mean that is off by e adds e^2 to the variance.
* y: xhat carries the errors of mean (times rstd) and rstd, the weight one rounding, the result o.
* dx: the two means have W + 32 roundings of the mean absolute term; everything is multiplied by rstd.
* dweight, dbias: (rows + 32) u of the sum of absolute terms, and xhat's own error.
"""
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


def make(rows, H, W, dtype, seed, par=True, shift=0.5):
    import torch

    gen = torch.Generator().manual_seed(seed)
    io = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    shape, p = ((rows, W), (W,)) if H == 1 else ((rows, H, W), (H, W))
    return {"x": (1.5 * n(*shape) + shift).to(io).cuda(), "dy": n(*shape).to(io).cuda(),
            "w": (1 + 0.2 * n(*p)).cuda() if par else None, "b": (0.1 * n(*p)).cuda() if par else None}


def check(z, what):
    import torch

    import selective_state_space_35_amd as ssm

    say(what)
    x, dy, w, b = z["x"], z["dy"], z["w"], z["b"]
    y, mean, rstd = ssm.ssm_layernorm_fwd(x, w, b, eps=EPS)
    d = ssm.ssm_layernorm_bwd(x, dy, mean, rstd, w, heads=None if w is not None or x.dim() == 2 else x.shape[1])
    torch.cuda.synchronize()
    f = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    X, DY, Wt, B = f(x), f(dy), f(w), f(b)
    W = X.shape[-1]
    o = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    one = torch.ones(d["dweight"].shape, dtype=torch.float64)
    Wt = one if Wt is None else Wt
    B = 0 * one if B is None else B
    m = X.mean(-1, keepdim=True)
    v = (X - m).square().mean(-1, keepdim=True)
    r = 1 / torch.sqrt(v + EPS)
    xh = (X - m) * r
    em = (W + 16) * U * X.abs().mean(-1, keepdim=True)
    er = r * (W + 32) * U + 0.5 * r ** 3 * em ** 2
    exh = r * em + (X - m).abs() * er + 4 * U * xh.abs()

    def ok(name, got, want, tol):
        over = ((f(got) - want).abs() / (tol * 1.01 + 1e-37)).max().item() if got.numel() else 0.0
        print(f"[layernorm] {what}: {name} at {over:.3f} of its bound", flush=True)
        assert over <= 1.0, f"{what}: {name} at {over} of its bound"

    ok("mean", mean, m[..., 0], em[..., 0])
    ok("rstd", rstd, r[..., 0], er[..., 0])
    ey = exh * Wt.abs() + 4 * U * (xh * Wt).abs() + 4 * U * B.abs()
    ok("y", y, xh * Wt + B, ey + o * (xh * Wt + B).abs())
    # the backward is given the forward's float mean and rstd: xhat of those
    M, R = f(mean).unsqueeze(-1), f(rstd).unsqueeze(-1)
    xh = (X - M) * R
    t = DY * Wt
    c1, c2 = t.mean(-1, keepdim=True), (t * xh).mean(-1, keepdim=True)
    a1, a2 = t.abs().mean(-1, keepdim=True), (t * xh).abs().mean(-1, keepdim=True)
    dx = R * (t - c1 - xh * c2)
    edx = R * (W + 32) * U * (t.abs() + a1 + xh.abs() * a2)
    ok("dx", d["dx"], dx, edx + o * dx.abs())
    n = X.shape[0]
    ok("dweight", d["dweight"], (DY * xh).sum(0), (n + 32) * U * (DY * xh).abs().sum(0))
    ok("dbias", d["dbias"], DY.sum(0), (n + 32) * U * DY.abs().sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 2, 3, 7, 8, 16, 31, 64, 65, 120, 128, 200, 256, 257, 512, 513, 768, 1000, 1024, 1025,
                               2048, 2049, 2560, 4096, 4100, 5120, 8192, 9001, 16384])
def test_widths(W, dtype):
    check(make(5, 1, W, dtype, W), f"layernorm W={W} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 3, 64, 1025, 3001])
def test_rows(rows, dtype):
    check(make(rows, 1, 96, dtype, rows), f"layernorm rows={rows} {dtype}")
    check(make(rows, 1, 1536, dtype, rows), f"layernorm rows={rows} W=1536 {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H,W", [(1, 2, 1), (7, 3, 64), (40, 24, 64), (700, 40, 128), (33, 5, 37), (9, 2, 1100),
                                      (3, 40, 72), (5000, 2, 8)])
def test_heads(rows, H, W, dtype):
    check(make(rows, H, W, dtype, rows + H), f"layernorm rows={rows} H={H} W={W} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_parameters(dtype):
    check(make(50, 1, 300, dtype, 1, par=False), f"layernorm no parameters {dtype}")
    check(make(50, 4, 32, dtype, 2, par=False), f"layernorm heads, no parameters {dtype}")


def test_far_from_zero():
    """A mean that is large against the spread: the variance is taken around the mean."""
    check(make(20, 1, 640, "f32", 3, shift=300.0), "layernorm shifted")


def test_unaligned_and_empty():
    import torch

    import selective_state_space_35_amd as ssm

    z = make(12, 1, 256, "bf16", 4)
    for k in ("x", "dy"):
        buf = torch.empty(z[k].numel() + 1, dtype=z[k].dtype, device="cuda")
        buf[1:] = z[k].reshape(-1)
        z[k] = buf[1:].view(12, 256)
    check(z, "layernorm unaligned")
    say("layernorm no rows")
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = ssm.ssm_layernorm_fwd(x, torch.ones(64, device="cuda"))
    d = ssm.ssm_layernorm_bwd(x, x, mean, rstd, torch.ones(64, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == (0, 64) and (d["dweight"] == 0).all() and (d["dbias"] == 0).all()


def test_rows_that_are_not_numbers_stay_alone():
    import torch

    import selective_state_space_35_amd as ssm

    for W in (64, 1001, 2560):
        z = make(9, 1, W, "f32", 5)
        y0, _, _ = ssm.ssm_layernorm_fwd(z["x"], z["w"], z["b"])
        z["x"][4, W // 2] = float("nan")
        z["x"][6, 0] = float("inf")
        say(f"layernorm not numbers W={W}")
        y, mean, rstd = ssm.ssm_layernorm_fwd(z["x"], z["w"], z["b"])
        dx = ssm.ssm_layernorm_bwd(z["x"], z["dy"], mean, rstd, z["w"], param_grads=False)["dx"]
        torch.cuda.synchronize()
        keep = [0, 1, 2, 3, 5, 7, 8]
        assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[4]).all() and torch.isnan(dx[4]).all()
        assert torch.isfinite(dx[keep]).all()


def test_deterministic_streams_and_graph():
    import torch

    import selective_state_space_35_amd as ssm

    z = make(3000, 6, 64, "bf16", 6)
    wide = make(600, 1, 2560, "bf16", 7)

    def work():
        out = []
        for t in (z, wide):
            y, m, r = ssm.ssm_layernorm_fwd(t["x"], t["w"], t["b"])
            d = ssm.ssm_layernorm_bwd(t["x"], t["dy"], m, r, t["w"])
            out += [y, m, r, d["dx"], d["dweight"], d["dbias"]]
        return out

    say("layernorm graph")
    eager = [t.clone() for t in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = work()
    same = work()
    torch.cuda.synchronize()
    for got in (other, same):
        assert all(torch.equal(a, b) for a, b in zip(eager, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for rep in range(3):
        for t in out:
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), f"replay {rep}"
        work()
