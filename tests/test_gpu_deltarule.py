"""The gated delta rule on the GPU, through the C ABI, against the float64 reference of tests/deltarule_ref.py (whose module
text derives the bounds)."""
import math

import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "bf16": "bfloat16"}


def make(b=2, L=70, H=4, G=2, Dk=40, Dv=24, dtype="bf16", seed=0, beta="sigmoid", gate=True, fixed=False, init=True,
         lengths=None, rate=0.1, close=0.0):
    """``close``: how much of one direction all keys of a head share (0: none, 1: they are the same)."""
    import torch

    gen = torch.Generator().manual_seed(seed)
    io = getattr(torch, DT[dtype])
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    k = unit(n(b, L, G, Dk))
    if close:
        k = unit((1 - close) * k + close * unit(n(b, 1, G, Dk)))
    # a key that rounding made longer than one would let errors grow: the bounds want |k| <= 1
    x = {"q": unit(n(b, L, G, Dk)), "k": k * (1 - 2.0 ** -7 if dtype == "bf16" else 1 - 2.0 ** -20), "v": n(b, L, H, Dv),
         "dy": n(b, L, H, Dv), "g": -rate * n(b, L, H).abs() if gate else None,
         "beta": None if beta is None else torch.sigmoid(n(b, L, H)) if beta == "sigmoid" else torch.full((b, L, H), float(beta))}
    x = {k: None if t is None else t.to(io).cuda() for k, t in x.items()}
    x["A"] = (-rate * n(H).abs()).cuda() if fixed else None
    x["initial_state"] = n(b, H, Dk, Dv).cuda() if init else None
    x["d_last_state"] = n(b, H, Dk, Dv).cuda() if init else None
    x["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    x["scale"] = Dk ** -0.5
    return x


def fwd(x, **kw):
    import selective_state_space_35_amd as ssm

    return ssm.ssm_deltarule_fwd(x["q"], x["k"], x["v"], beta=x["beta"], g=x["g"], A=x["A"], scale=x["scale"],
                                 lengths=x["lengths"], initial_state=x["initial_state"], **kw)


def bwd(x):
    import selective_state_space_35_amd as ssm

    return ssm.ssm_deltarule_bwd(x["q"], x["k"], x["v"], x["dy"], beta=x["beta"], g=x["g"], A=x["A"], scale=x["scale"],
                                 lengths=x["lengths"], initial_state=x["initial_state"], d_last_state=x["d_last_state"])


def check(x, what, backward=True):
    import torch

    from tests import deltarule_ref as ref

    say(what)
    y, last = fwd(x)
    torch.cuda.synchronize()
    want, V = ref.forward(x)
    ref.within(y, want["y"], V["y"], "y", x, what)
    ref.within(last, want["last_state"], V["last_state"], "last_state", x, what)
    if not backward:
        return
    say(what + ", backward")
    d = bwd(x)
    torch.cuda.synchronize()
    want, V = ref.backward(x)
    for name, given in (("dg", "g"), ("dbeta", "beta"), ("d_initial_state", "initial_state")):
        assert (d[name] is None) == (x[given] is None)
    for name, t in d.items():
        if t is not None:
            ref.within(t, want[name], V[name], name, x, what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 47, 49, 63, 64, 65, 127, 128, 129, 200, 513])
def test_lengths(L, dtype):
    check(make(b=1, L=L, H=2, G=2, Dk=64, Dv=64, dtype=dtype, seed=L), f"deltarule L={L} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 5), (16, 16), (33, 31), (40, 72), (64, 128), (128, 64), (128, 128),
                                   (100, 127), (127, 4), (8, 120), (24, 80)])
def test_widths(Dk, Dv, dtype):
    check(make(b=1, L=150, H=3, G=3, Dk=Dk, Dv=Dv, dtype=dtype, seed=Dk + Dv), f"deltarule Dk={Dk} Dv={Dv} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 1), (6, 2), (6, 3), (6, 6), (17, 17), (8, 2)])
def test_groups_of_heads(H, G, dtype):
    check(make(b=2, L=90, H=H, G=G, Dk=32, Dv=48, dtype=dtype, seed=H + G), f"deltarule H={H} G={G} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,fixed,init", [(False, False, False), (False, True, False), (False, True, True),
                                             (True, False, False), (True, True, True)])
def test_decays_and_states(gate, fixed, init, dtype):
    check(make(gate=gate, fixed=fixed, init=init, dtype=dtype, L=140, seed=9), f"deltarule gate={gate} A={fixed} init={init} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("beta", [None, 0.0, 1.0, 2.0, 1e-3, 1e-30])
@pytest.mark.parametrize("close", [0.0, 0.7, 1.0])
def test_strengths_and_close_keys(beta, close, dtype):
    """From no write at all to one that turns the state around, with keys that differ and keys that are all the same."""
    check(make(L=130, beta=beta, close=close, dtype=dtype, gate=close != 1.0, seed=3), f"deltarule beta={beta} close={close} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_beta_of_zero_writes_nothing(dtype):
    import torch

    x = make(L=75, dtype=dtype, seed=8, gate=False)
    x["beta"][:, 10:70] = 0
    y, last = fwd(x)
    d = bwd(x)
    x2 = dict(x, v=x["v"].clone())
    x2["v"][:, 10:70] = 5.0
    y2, last2 = fwd(x2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2)
    assert (d["dv"][:, 10:70] == 0).all() and (d["dbeta"][:, 10:70] != 0).any()
    check(x, f"deltarule beta zero in places {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,lengths", [(70, [70, 0, 1]), (130, [64, 65, 129]), (5, [-3, 9, 5]), (300, [299, 63, 128])])
def test_padded_batch(L, lengths, dtype):
    """Tokens behind a row's length may hold anything: they are not read, and their rows are zero."""
    import torch

    x = make(b=3, L=L, lengths=lengths, dtype=dtype, seed=L)
    n = [min(max(v, 0), L) for v in lengths]
    clean = {k: x[k].clone() for k in ("q", "k", "v", "g", "beta", "dy")}
    for k in clean:
        for i in range(3):
            x[k][i, n[i]:] = float("nan") if i != 1 else float("inf")
            clean[k][i, n[i]:] = 0
    what = f"deltarule padded L={L} {lengths} {dtype}"
    say(what)
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    for i in range(3):
        assert (y[i, n[i]:] == 0).all()
        for k in ("dq", "dk", "dv", "dg", "dbeta"):
            assert (d[k][i, n[i]:] == 0).all(), k
        if n[i] == 0:
            assert torch.equal(last[i], x["initial_state"][i])
            assert torch.equal(d["d_initial_state"][i], x["d_last_state"][i])
    check(dict(x, **clean), what)
    y2, last2 = fwd(dict(x, **clean))
    assert torch.equal(y, y2) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [1e-4, 1.0, 6.0])
def test_slow_and_fast_decays(rate, dtype):
    """From a memory of the whole sequence to one of less than a token."""
    check(make(L=200, rate=rate, dtype=dtype, seed=4), f"deltarule rate={rate} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-math.inf, -3e4, -200.0])
def test_resets(value, dtype):
    """A gate of minus infinity (or far below what float's exp can tell from it) drops the state: documents that follow
    each other in a row are separate ones, in their gradients too."""
    import torch

    from tests import deltarule_ref as ref

    x = make(L=210, dtype=dtype, seed=6)
    cuts = (0, 1, 37, 64, 65, 66, 130, 209)
    for t in cuts:
        x["g"][:, t] = value
    check(x, f"deltarule reset {value} {dtype}", backward=False)
    y, _ = fwd(x)
    cut = {k: x[k][:, 66:130].contiguous() for k in ("q", "k", "v", "g", "beta", "dy")}
    sub = dict(x, initial_state=None, d_last_state=None, **cut)
    want, V = ref.forward(sub)
    ref.within(y[:, 66:130], want["y"], V["y"], "y", sub, f"a document alone {value} {dtype}")
    d = bwd(x)
    torch.cuda.synchronize()
    for t in cuts:
        assert (d["dg"][:, t] == 0).all()
    want, V = ref.backward(x)
    for name, t in d.items():
        ref.within(t, want[name], V[name], name, x, f"deltarule reset {value} {dtype}")
    # what follows a reset does not come into the gradients before it
    z = dict(x, v=x["v"].clone(), dy=x["dy"].clone())
    z["v"][:, 130:] *= 1e4
    z["dy"][:, 130:] *= 1e4
    d2 = bwd(z)
    torch.cuda.synchronize()
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        ref.within(d2[name][:, 66:130], want[name][:, 66:130], V[name][:, 66:130], name, x, f"before a loud document {value} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "g"])
def test_what_is_not_finite_does_not_reach_back(name, bad, dtype):
    """A token's value that is no number reaches its own output and later ones, bit for bit no earlier token's and no other
    head's; one of v its own column alone, one of q its own row."""
    import torch

    x = make(b=1, L=200, H=4, G=4, Dk=40, Dv=72, dtype=dtype, seed=21, rate=0.05)
    say(f"deltarule {name} = {bad} {dtype}")
    y0, _ = fwd(x)
    others = [0, 2, 3]
    col = [j for j in range(72) if j != 5]
    for t in (0, 17, 70, 127, 199):
        z = dict(x, **{name: x[name].clone()})
        z[name][(0, t, 1) if name in ("beta", "g") else (0, t, 1, 5)] = bad
        y, last = fwd(z)
        torch.cuda.synchronize()
        assert torch.equal(y[0, :t], y0[0, :t]), t
        assert torch.equal(y[0, :, others], y0[0, :, others])
        if name == "v":
            assert torch.equal(y[0, :, 1][:, col], y0[0, :, 1][:, col])
            assert not torch.isfinite(y[0, t:, 1, 5]).any() and torch.isfinite(last[0, 1][:, col]).all()
            assert not torch.isfinite(last[0, 1, :, 5]).any()
        elif name == "q":
            assert torch.equal(y[0, t + 1:], y0[0, t + 1:]) and not torch.isfinite(y[0, t, 1]).any()
            assert torch.isfinite(last).all()
        else:
            assert not torch.isfinite(y[0, t:, 1]).any() and not torch.isfinite(last[0, 1]).any()
        assert torch.isfinite(last[0, others]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv,G", [(64, 64, 4), (128, 128, 4), (40, 72, 2), (33, 31, 1), (100, 127, 4), (1, 1, 4), (128, 3, 2)])
def test_tokens(Dk, Dv, G, dtype):
    """The step for one token, over a short sequence, is the sequence form's."""
    import torch

    import selective_state_space_35_amd as ssm
    from tests import deltarule_ref as ref

    x = make(b=3, L=6, H=4, G=G, Dk=Dk, Dv=Dv, dtype=dtype, seed=Dk, fixed=True)
    say(f"deltarule tokens Dk={Dk} Dv={Dv} {dtype}")
    state = x["initial_state"].clone()
    ys = []
    for t in range(6):
        q, k, v, g, beta = (x[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta"))
        ys.append(ssm.ssm_deltarule_update(state, q, k, v, beta=beta, g=g, A=x["A"], scale=x["scale"]))
    torch.cuda.synchronize()
    want, V = ref.forward(x)
    ref.within(torch.stack(ys, 1), want["y"], V["y"], "y", x, "tokens")
    ref.within(state, want["last_state"], V["last_state"], "last_state", x, "tokens")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_of_rows_that_have_ended(dtype):
    import torch

    import selective_state_space_35_amd as ssm

    x = make(b=4, L=1, H=3, G=3, Dk=48, Dv=40, dtype=dtype, lengths=[1, 0, -2, 5])
    q, k, v, g, beta = (x[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta"))
    for t in (q, k, v, g, beta):
        t[1:3] = float("nan")
    state = x["initial_state"].clone()
    y = ssm.ssm_deltarule_update(state, q, k, v, beta=beta, g=g, lengths=x["lengths"])
    torch.cuda.synchronize()
    assert torch.equal(state[1:3], x["initial_state"][1:3]) and (y[1:3] == 0).all()
    assert torch.isfinite(y).all() and not torch.equal(state[0], x["initial_state"][0]) and (y[3] != 0).any()


def test_empty_calls():
    import torch

    import selective_state_space_35_amd as ssm

    x = make(b=2, L=0)
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 4, 24) and torch.equal(last, x["initial_state"])
    assert torch.equal(d["d_initial_state"], x["d_last_state"]) and d["dq"].shape == (2, 0, 2, 40)
    y, last = fwd(make(b=2, L=0, init=False))
    torch.cuda.synchronize()
    assert (last == 0).all()
    fwd(make(b=0, L=5)), bwd(make(b=0, L=5))
    z = torch.zeros(0, 2, 8, device="cuda")
    assert ssm.ssm_deltarule_update(torch.zeros(0, 4, 8, 8, device="cuda"), z, z, torch.zeros(0, 4, 8, device="cuda")).shape == (0, 4, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_asking_for_less_changes_nothing(dtype):
    import torch

    x = make(L=150, dtype=dtype, seed=12)
    y, last = fwd(x)
    y2, none = fwd(x, return_last_state=False)
    d = bwd(x)
    d2 = bwd(x)
    torch.cuda.synchronize()
    assert none is None and torch.equal(y, y2)
    for n, t in d.items():
        assert torch.equal(t, d2[n]), n
    # whole sequences are joined parts of them
    a = {k: t[:, :90].contiguous() if k in ("q", "k", "v", "g", "beta") else t for k, t in x.items()}
    b = {k: t[:, 90:].contiguous() if k in ("q", "k", "v", "g", "beta") else t for k, t in x.items()}
    ya, mid = fwd(a)
    yb, end = fwd(dict(b, initial_state=mid))
    from tests import deltarule_ref as ref
    want, V = ref.forward(x)
    ref.within(torch.cat([ya, yb], 1), want["y"], V["y"], "y", x, "joined")
    ref.within(end, want["last_state"], V["last_state"], "last_state", x, "joined")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 40])
def test_unaligned_tensors(dtype, D):
    """Tensors that begin one element behind an aligned address."""
    import torch

    x = make(b=2, L=100, H=4, G=4, Dk=D, Dv=D, dtype=dtype, seed=5)
    y0, l0 = fwd(x)
    d0 = bwd(x)
    for k in ("q", "k", "v", "g", "beta", "dy", "initial_state"):
        room = torch.empty(x[k].numel() + 1, dtype=x[k].dtype, device="cuda")
        room[1:] = x[k].reshape(-1)
        x[k] = room[1:].view(x[k].shape)
    say(f"deltarule unaligned D={D} {dtype}")
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(last, l0)
    for n in d:
        assert torch.equal(d[n], d0[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_heads_and_rows(dtype):
    """More workgroups than the chip holds at once."""
    check(make(b=9, L=70, H=40, G=8, Dk=16, Dv=80, dtype=dtype, seed=31), f"deltarule many {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_and_stream(dtype):
    """Captured with a workspace of the caller's, on another stream, and replayed with other inputs."""
    import torch

    import selective_state_space_35_amd as ssm

    x = make(L=150, dtype=dtype, seed=17, lengths=[150, 77])
    names = ("q", "k", "v", "g", "beta", "dy")
    more = [make(L=150, dtype=dtype, seed=s) for s in (18, 19, 20)]
    say(f"deltarule graph {dtype}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd(x), bwd(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    tok = [x[n][:, 0].contiguous() for n in ("q", "k", "v", "beta", "g")]
    state = x["initial_state"].clone()
    with torch.cuda.graph(graph):
        y, last = fwd(x)
        d = bwd(x)
        yt = ssm.ssm_deltarule_update(state, tok[0], tok[1], tok[2], beta=tok[3], g=tok[4])
    for m in more:
        for n in names:
            x[n].copy_(m[n])
        state.copy_(x["initial_state"])
        y0, l0 = fwd(x)
        d0 = bwd(x)
        s0 = x["initial_state"].clone()
        t0 = ssm.ssm_deltarule_update(s0, tok[0], tok[1], tok[2], beta=tok[3], g=tok[4])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(last, l0) and torch.equal(yt, t0) and torch.equal(state, s0)
        for n in d:
            assert torch.equal(d[n], d0[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,Dk", [(32, 8, 40), (12, 2, 72)])
def test_heads_that_share_one_workgroup(H, G, Dk, dtype):
    """So many chunks that the backward takes the heads of a group, or some of them, one after the other."""
    b, L = (16, 520) if G == 8 else (16, 200 if dtype == "f32" else 400)
    check(make(b=b, L=L, H=H, G=G, Dk=Dk, Dv=8, dtype=dtype, seed=33, lengths=[L - 3 * i for i in range(b)]),
          f"deltarule shared H={H} G={G} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,L,H,G,Dk,Dv,lengths", [(1, 1500, 2, 1, 64, 48, None), (2, 2100, 1, 1, 128, 128, [2100, 700]),
                                                   (3, 900, 2, 2, 40, 72, [0, 1, 899]), (1, 3000, 5, 5, 16, 16, None),
                                                   (1, 640, 1, 1, 100, 24, [513])])
def test_cut_sequences(b, L, H, G, Dk, Dv, lengths, dtype):
    """Few heads and a long sequence: the sequence is cut, and its pieces' states are joined by their maps."""
    check(make(b=b, L=L, H=H, G=G, Dk=Dk, Dv=Dv, dtype=dtype, rate=0.01, seed=L, lengths=lengths),
          f"deltarule cut b={b} L={L} H={H} Dk={Dk} Dv={Dv} {lengths} {dtype}")
