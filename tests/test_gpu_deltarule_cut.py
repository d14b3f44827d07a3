"""The gated delta rule on sequences that are cut into segments, whose entering states come from the parts' own states and
maps: values that are not finite, resets and lengths inside parts, at their borders and in the last segment, heads to 64 and
above."""
import math

import pytest

from tests import deltarule_plan as plan
from tests.gpu_common import say
from tests.test_gpu_deltarule import bwd, check, fwd, make

pytestmark = pytest.mark.gpu


def borders(b, L, H, Dk, Dv, dtype):
    """First tokens of parts and of the last segment; asserts that the sequence is cut."""
    segs, parts, pc, n_parts = plan.cut(b, L, H, Dk, Dv, dtype)
    assert segs > 1 and n_parts > 1
    step = pc * plan.CHUNK[dtype]
    return step, 2 * step, n_parts * step


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "g"])
@pytest.mark.parametrize("L,Dk,Dv", [(1500, 40, 72), (1500, 128, 72), (200, 128, 72), (130, 100, 128)])
def test_what_is_not_finite_does_not_reach_back(L, Dk, Dv, name, bad, dtype):
    """A token's value that is no number reaches its own output and later ones, bit for bit no earlier token's and no other
    head's; one of v its own column alone, one of q its own row."""
    import torch

    x = make(b=1, L=L, H=4, G=4, Dk=Dk, Dv=Dv, dtype=dtype, seed=21, rate=0.05)
    what = f"deltarule {name} = {bad} L={L} Dk={Dk} Dv={Dv} {dtype}"
    say(what)
    first, second, last_segment = borders(1, L, 4, Dk, Dv, dtype) if L > 1000 else (17, 70, 127)
    y0, _ = fwd(x)
    others = [0, 2, 3]
    col = [j for j in range(Dv) if j != 69]
    for t in (0, first - 1, first, second + 3, last_segment - 1, last_segment, L - 1):
        z = dict(x, **{name: x[name].clone()})
        z[name][(0, t, 1) if name in ("beta", "g") else (0, t, 1, 69 if name == "v" else 5)] = bad
        y, last = fwd(z)
        torch.cuda.synchronize()
        assert torch.equal(y[0, :t], y0[0, :t]), t
        assert torch.equal(y[0, :, others], y0[0, :, others]), t
        if name == "v":
            assert torch.equal(y[0, :, 1][:, col], y0[0, :, 1][:, col]), t
            assert not torch.isfinite(y[0, t:, 1, 69]).any() and torch.isfinite(last[0, 1][:, col]).all(), t
            assert not torch.isfinite(last[0, 1, :, 69]).any(), t
        elif name == "q":
            assert torch.equal(y[0, t + 1:], y0[0, t + 1:]) and not torch.isfinite(y[0, t, 1]).any(), t
            assert torch.isfinite(last).all(), t
        else:
            assert not torch.isfinite(y[0, t:, 1]).any() and not torch.isfinite(last[0, 1]).any(), t
        assert torch.isfinite(last[0, others]).all(), t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-math.inf, -3e4, -200.0])
@pytest.mark.parametrize("Dk,Dv", [(40, 24), (96, 24)])
def test_resets(Dk, Dv, value, dtype):
    """Documents that follow each other in a row that is cut are separate ones, in their gradients too."""
    import torch

    from tests import deltarule_ref as ref

    L = 1500
    first, second, last_segment = borders(2, L, 4, Dk, Dv, dtype)
    x = make(L=L, Dk=Dk, Dv=Dv, dtype=dtype, seed=6, rate=0.02)
    cuts = sorted({0, 1, first - 1, first, second + 5, last_segment - 40, last_segment, last_segment + 33, L - 1})
    for t in cuts:
        x["g"][:, t] = value
    what = f"deltarule cut, reset {value} Dk={Dk} {dtype}"
    check(x, what, backward=False)
    y, _ = fwd(x)
    a, e = first, second + 5
    sub = dict(x, initial_state=None, d_last_state=None, **{k: x[k][:, a:e].contiguous() for k in ("q", "k", "v", "g", "beta", "dy")})
    want, V = ref.forward(sub)
    ref.within(y[:, a:e], want["y"], V["y"], "y", sub, what + ", a document alone")
    d = bwd(x)
    torch.cuda.synchronize()
    for t in cuts:
        assert (d["dg"][:, t] == 0).all()
    want, V = ref.backward(x)
    for name, t in d.items():
        ref.within(t, want[name], V[name], name, x, what)
    # what follows a reset does not come into the gradients before it
    z = dict(x, v=x["v"].clone(), dy=x["dy"].clone())
    z["v"][:, e:] *= 1e4
    z["dy"][:, e:] *= 1e4
    d2 = bwd(z)
    torch.cuda.synchronize()
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        ref.within(d2[name][:, a:e], want[name][:, a:e], V[name][:, a:e], name, x, what + ", before a loud document")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,L,H,G,Dk,Dv,lengths", [(1, 1700, 1, 1, 100, 24, [513]), (3, 1500, 3, 1, 72, 100, [1500, 0, 700]),
                                                   (2, 1400, 4, 2, 33, 31, [1, 1399])])
def test_lengths_in_parts(b, L, H, G, Dk, Dv, lengths, dtype):
    borders(b, L, H, Dk, Dv, dtype)
    check(make(b=b, L=L, H=H, G=G, Dk=Dk, Dv=Dv, dtype=dtype, rate=0.01, seed=L, lengths=lengths),
          f"deltarule cut b={b} L={L} H={H} Dk={Dk} Dv={Dv} {lengths} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_of_a_cut_sequence_is_not_read(dtype):
    import torch

    x = make(b=2, L=1500, H=2, G=2, Dk=72, Dv=40, lengths=[900, 64], dtype=dtype, seed=9)
    borders(2, 1500, 2, 72, 40, dtype)
    say(f"deltarule cut, padding {dtype}")
    y0, l0 = fwd(x)
    d0 = bwd(x)
    for k in ("q", "k", "v", "g", "beta", "dy"):
        x[k][0, 900:] = float("nan")
        x[k][1, 64:] = float("inf")
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(last, l0)
    for k in d:
        assert torch.equal(d[k], d0[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph(dtype):
    """Captured calls of a cut sequence, replayed with other inputs."""
    import torch

    x = make(b=1, L=1500, H=2, G=1, Dk=72, Dv=40, dtype=dtype, seed=17)
    borders(1, 1500, 2, 72, 40, dtype)
    say(f"deltarule cut, graph {dtype}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd(x), bwd(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = fwd(x)
        d = bwd(x)
    for seed in (18, 19, 20):
        m = make(b=1, L=1500, H=2, G=1, Dk=72, Dv=40, dtype=dtype, seed=seed)
        for k in ("q", "k", "v", "g", "beta", "dy", "initial_state", "d_last_state"):
            x[k].copy_(m[k])
        y0, l0 = fwd(x)
        d0 = bwd(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(last, l0)
        for k in d:
            assert torch.equal(d[k], d0[k]), k
