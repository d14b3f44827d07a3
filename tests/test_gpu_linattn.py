"""Linear attention with a decay for each head on the GPU, through the C ABI, against the float64
reference of tests/linattn_ref.py (whose module text derives the bounds)."""
import math

import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "bf16": "bfloat16"}


def make(b=2, L=70, H=4, G=2, Dk=40, Dv=24, dtype="bf16", seed=0, gate=True, fixed=False, init=True, lengths=None,
         rate=0.1):
    import torch

    gen = torch.Generator().manual_seed(seed)
    io = getattr(torch, DT[dtype])
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = {"q": n(b, L, G, Dk), "k": n(b, L, G, Dk), "v": n(b, L, H, Dv), "dy": n(b, L, H, Dv),
         "g": -rate * n(b, L, H).abs() if gate else None}
    x = {k: None if t is None else t.to(io).cuda() for k, t in x.items()}
    x["A"] = (-rate * n(H).abs()).cuda() if fixed else None
    x["initial_state"] = n(b, H, Dk, Dv).cuda() if init else None
    x["d_last_state"] = n(b, H, Dk, Dv).cuda() if init else None
    x["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    x["scale"] = Dk ** -0.5
    return x


def fwd(x, **kw):
    import selective_state_space_35_amd as ssm

    return ssm.ssm_linattn_fwd(x["q"], x["k"], x["v"], g=x["g"], A=x["A"], scale=x["scale"], lengths=x["lengths"],
                               initial_state=x["initial_state"], **kw)


def bwd(x):
    import selective_state_space_35_amd as ssm

    return ssm.ssm_linattn_bwd(x["q"], x["k"], x["v"], x["dy"], g=x["g"], A=x["A"], scale=x["scale"],
                               lengths=x["lengths"], initial_state=x["initial_state"], d_last_state=x["d_last_state"])


def check(x, what, backward=True):
    import torch

    from tests import linattn_ref as ref

    say(what)
    y, last = fwd(x)
    torch.cuda.synchronize()
    want, mag = ref.forward(x), ref.forward(x, absolute=True)
    ref.within(y, want["y"], mag["y"], "y", x, what)
    ref.within(last, want["last_state"], mag["last_state"], "last_state", x, what)
    if not backward:
        return
    say(what + ", backward")
    d = bwd(x)
    torch.cuda.synchronize()
    want, mag = ref.backward(x), ref.backward(x, absolute=True)
    assert (d["dg"] is None) == (x["g"] is None) and (d["d_initial_state"] is None) == (x["initial_state"] is None)
    for name, t in d.items():
        if t is not None:
            ref.within(t, want[name], mag[name], name, x, what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 511, 513])
def test_lengths(L, dtype):
    check(make(b=1, L=L, H=2, G=2, Dk=64, Dv=64, dtype=dtype, seed=L), f"linattn L={L} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 5), (16, 16), (33, 31), (40, 72), (64, 128), (128, 64), (128, 128),
                                   (100, 127), (127, 4), (8, 120)])
def test_widths(Dk, Dv, dtype):
    check(make(b=1, L=150, H=3, G=3, Dk=Dk, Dv=Dv, dtype=dtype, seed=Dk + Dv), f"linattn Dk={Dk} Dv={Dv} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 1), (6, 2), (6, 3), (6, 6), (17, 17), (8, 2)])
def test_groups_of_heads(H, G, dtype):
    check(make(b=2, L=90, H=H, G=G, Dk=32, Dv=48, dtype=dtype, seed=H + G), f"linattn H={H} G={G} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,fixed,init", [(False, False, False), (False, True, False), (False, True, True),
                                             (True, False, False), (True, True, True)])
def test_decays_and_states(gate, fixed, init, dtype):
    check(make(gate=gate, fixed=fixed, init=init, dtype=dtype, L=140, seed=9), f"linattn gate={gate} A={fixed} init={init} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,lengths", [(70, [70, 0, 1]), (130, [64, 65, 129]), (5, [-3, 9, 5]), (300, [299, 63, 128])])
def test_padded_batch(L, lengths, dtype):
    """Tokens behind a row's length may hold anything: they are not read, and their rows are zero."""
    import torch

    x = make(b=3, L=L, lengths=lengths, dtype=dtype, seed=L)
    n = [min(max(v, 0), L) for v in lengths]
    clean = {k: None if t is None else t.clone() for k, t in x.items() if k in ("q", "k", "v", "g", "dy")}
    for k in clean:
        for i in range(3):
            x[k][i, n[i]:] = float("nan") if i != 1 else float("inf")
            clean[k][i, n[i]:] = 0
    what = f"linattn padded L={L} {lengths} {dtype}"
    say(what)
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    for i in range(3):
        assert (y[i, n[i]:] == 0).all()
        for k in ("dq", "dk", "dv", "dg"):
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
    check(make(L=200, rate=rate, dtype=dtype, seed=4), f"linattn rate={rate} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-math.inf, -3e4, -200.0])
def test_resets(value, dtype):
    """A gate of minus infinity (or far below what float's exp can tell from it) drops the state: documents
    that follow each other in a row are separate ones."""
    import torch

    from tests import linattn_ref as ref

    x = make(L=210, dtype=dtype, seed=6)
    for t in (0, 1, 37, 64, 65, 66, 130, 209):
        x["g"][:, t] = value
    check(x, f"linattn reset {value} {dtype}", backward=False)
    y, _ = fwd(x)
    cut = {k: t[:, 66:130].contiguous() for k, t in x.items() if k in ("q", "k", "v", "g")}
    sub = dict(x, initial_state=None, **cut)
    want, mag = ref.forward(sub), ref.forward(sub, absolute=True)
    ref.within(y[:, 66:130], want["y"], mag["y"], "y", sub, f"a document alone {value} {dtype}")
    d = bwd(x)
    torch.cuda.synchronize()
    want, mag = ref.backward(x), ref.backward(x, absolute=True)
    for name, t in d.items():
        ref.within(t, want[name], mag[name], name, x, f"linattn reset {value} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_segments(dtype):
    """Few heads and a long sequence: the sequence is cut and its pieces' states are joined."""
    check(make(b=1, L=1500, H=2, G=1, Dk=64, Dv=48, dtype=dtype, rate=0.01, seed=2), f"linattn segments {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_what_is_not_finite_does_not_reach_back(name, bad, dtype):
    """A token's value that is no number reaches its own output and later ones, bit for bit no earlier token's; in the
    backward (through dy) no later token's dq and dk.  What stands in v's place (v in y, dy in dv) may reach the other
    tokens of its step, 63 (f32: 31) at most, in its own column, as documented: beyond them it is equality too."""
    import torch

    x = make(b=1, L=230, H=4, G=4, Dk=40, Dv=72, dtype=dtype, seed=21, rate=0.05)
    say(f"linattn {name} = {bad} {dtype}")
    step = 31 if dtype == "f32" else 63
    y0, _ = fwd(x)
    d0 = bwd(x)
    others = [0, 2, 3]
    col = [j for j in range(72) if j != 5]
    for t in (0, 70, 127, 229):
        z = dict(x, **{name: x[name].clone()})
        z[name][0, t, 1, 5] = bad
        y, last = fwd(z)
        torch.cuda.synchronize()
        before = max(t - step, 0) if name == "v" else t
        assert torch.equal(y[0, :before], y0[0, :before]), t
        assert torch.equal(y[0, :, others], y0[0, :, others])
        if name == "v":
            assert torch.equal(y[0, :t, 1][:, col], y0[0, :t, 1][:, col])
            assert not torch.isfinite(y[0, t:, 1, 5]).any() and torch.isfinite(y[0, :, 1, col]).all()
        if name == "q":
            assert torch.equal(y[0, t + 1:], y0[0, t + 1:]) and not torch.isfinite(y[0, t, 1]).any()
        if name != "q":
            assert not torch.isfinite(last[0, 1]).all() and torch.isfinite(last[0, others]).all()
        z = dict(x, dy=x["dy"].clone())
        z["dy"][0, t, 1, 5] = bad
        d = bwd(z)
        torch.cuda.synchronize()
        assert torch.equal(d["dk"][0, t + 1:], d0["dk"][0, t + 1:]), t
        assert torch.equal(d["dv"][0, t + 1 + step:], d0["dv"][0, t + 1 + step:]), t
        assert torch.equal(d["dv"][0, t + 1:, 1][:, col], d0["dv"][0, t + 1:, 1][:, col]), t
        assert torch.equal(d["dq"][0, :t], d0["dq"][0, :t]) and torch.equal(d["dq"][0, t + 1:], d0["dq"][0, t + 1:])


def test_unaligned_rows():
    """Tensors that start in the middle of a 16-byte unit."""
    import torch

    x = make(L=100, Dk=32, Dv=64)
    for k in ("q", "k", "v", "dy"):
        buf = torch.empty(x[k].numel() + 1, dtype=x[k].dtype, device="cuda")
        buf[1:] = x[k].reshape(-1)
        x[k] = buf[1:].view(x[k].shape)
    check(x, "linattn unaligned")


def test_empty_sequence():
    import torch

    x = make(L=0)
    say("linattn L=0")
    y, last = fwd(x)
    d = bwd(x)
    assert y.shape == (2, 0, 4, 24) and torch.equal(last, x["initial_state"])
    assert torch.equal(d["d_initial_state"], x["d_last_state"]) and d["dq"].shape == x["q"].shape
    x["initial_state"] = None
    _, last = fwd(x)
    assert (last == 0).all()
    y, last = fwd(make(b=0))
    assert y.shape[0] == 0 and last.shape[0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_continue(dtype):
    """A sequence in two calls, the second from the first's state, is the sequence in one."""
    from tests import linattn_ref as ref

    x = make(L=333, dtype=dtype, seed=8)
    say(f"linattn pieces {dtype}")
    cut = lambda a, b: dict(x, **{k: x[k][:, a:b].contiguous() for k in ("q", "k", "v", "g")})  # noqa: E731
    y1, s1 = fwd(cut(0, 100))
    y2, s2 = fwd(dict(cut(100, 333), initial_state=s1))
    want, mag = ref.forward(x), ref.forward(x, absolute=True)
    ref.within(y1, want["y"][:, :100], mag["y"][:, :100], "y", x, "first piece")
    ref.within(y2, want["y"][:, 100:], mag["y"][:, 100:], "y", x, "second piece")
    ref.within(s2, want["last_state"], mag["last_state"] * 2, "last_state", x, "second piece")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,H,G,Dk,Dv", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (2, 6, 6, 128, 128), (2, 3, 1, 33, 70),
                                         (5, 2, 2, 5, 3), (2, 2, 2, 100, 4)])
def test_update(b, H, G, Dk, Dv, dtype):
    """Tokens one at a time: outputs and state of the recurrence; rows of length zero take no step."""
    import torch

    import selective_state_space_35_amd as ssm
    from tests import linattn_ref as ref

    T = 6
    x = make(b=b, L=T, H=H, G=G, Dk=Dk, Dv=Dv, dtype=dtype, fixed=True, seed=b + Dk)
    what = f"linattn update b{b} H{H} G{G} Dk{Dk} Dv{Dv} {dtype}"
    say(what)
    state = x["initial_state"].clone()
    ys = [ssm.ssm_linattn_update(state, x["q"][:, t].contiguous(), x["k"][:, t].contiguous(), x["v"][:, t].contiguous(),
                                 g=x["g"][:, t].contiguous(), A=x["A"], scale=x["scale"]) for t in range(T)]
    torch.cuda.synchronize()
    want, mag = ref.forward(x), ref.forward(x, absolute=True)
    ref.within(torch.stack(ys, 1), want["y"], mag["y"], "y", x, what)
    ref.within(state, want["last_state"], mag["last_state"], "last_state", dict(x, v=x["v"].float()), what)
    # a padded batch: rows 1.. wait
    lengths = torch.zeros(b, dtype=torch.int32, device="cuda")
    lengths[0] = 1
    before = state.clone()
    y = ssm.ssm_linattn_update(state, x["q"][:, 0].contiguous(), x["k"][:, 0].contiguous(), x["v"][:, 0].contiguous(),
                               A=x["A"], lengths=lengths)
    assert torch.equal(state[1:], before[1:]) and (y[1:] == 0).all()
    assert not torch.equal(state[0], before[0])


def test_update_of_an_unaligned_state():
    import torch

    import selective_state_space_35_amd as ssm

    x = make(b=2, L=1, H=4, G=4, Dk=32, Dv=64)
    tok = [x[k][:, 0].contiguous() for k in ("q", "k", "v")]
    a = x["initial_state"].clone()
    buf = torch.empty(a.numel() + 1, device="cuda")
    buf[1:] = a.reshape(-1)
    b = buf[1:].view(a.shape)
    say("linattn update unaligned")
    ya, yb = ssm.ssm_linattn_update(a, *tok), ssm.ssm_linattn_update(b, *tok)
    # the two forms add the readout's 32 products in different orders
    assert torch.equal(a, b)
    assert ((ya.float() - yb.float()).abs() <= 2.0 ** -7 * ya.float().abs() + 1e-4).all()


def test_deterministic_and_on_another_stream():
    import torch

    x = make(b=2, L=700, H=8, G=2, Dk=64, Dv=128, seed=3)
    say("linattn determinism")
    y, last = fwd(x)
    d = bwd(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, last2 = fwd(x)
        d2 = bwd(x)
    y3, last3 = fwd(x)  # at the same time on the first stream
    d3 = bwd(x)
    torch.cuda.synchronize()
    for yy, ll, dd in ((y2, last2, d2), (y3, last3, d3)):
        assert torch.equal(y, yy) and torch.equal(last, ll)
        assert all(torch.equal(d[k], dd[k]) for k in d)


def test_workspace_of_the_library_and_of_the_caller():
    """The C entry points with no workspace, with one, and with one that is too small."""
    import torch

    import selective_state_space_35_amd as ssm

    x = make(b=1, L=1500, H=2, G=1, Dk=64, Dv=64, init=False)
    say("linattn workspaces")
    y, last = fwd(x)
    d = bwd(x)
    lib = ssm.load_library()
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    dims = (1, 1500, 2, 1, 64, 64, 1)
    y2, last2 = torch.empty_like(y), torch.empty_like(last)
    d2 = {k: torch.empty_like(t) for k, t in d.items() if t is not None}

    def both(ws, n):
        a = lib.ssm_linattn_fwd(p(x["q"]), p(x["k"]), p(x["v"]), p(x["g"]), None, None, x["scale"], None, p(y2),
                                p(last2), *dims, ws, n, st)
        b = lib.ssm_linattn_bwd(p(x["q"]), p(x["k"]), p(x["v"]), p(x["g"]), None, None, x["scale"], None, p(x["dy"]), None,
                                p(d2["dq"]), p(d2["dk"]), p(d2["dv"]), p(d2["dg"]), None, *dims, ws, n, st)
        return a, b

    need = ssm.ssm_linattn_workspace(1, 1500, 2, 1, 64, 64, "bf16", True)
    ws = torch.empty(max(need, ssm.ssm_linattn_workspace(1, 1500, 2, 1, 64, 64, "bf16")), dtype=torch.uint8, device="cuda")
    for args in ((None, 0), (ws.data_ptr(), ws.numel())):
        for t in (y2, last2, *d2.values()):
            t.fill_(7)
        assert both(*args) == (0, 0)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(last, last2) and all(torch.equal(d[k], d2[k]) for k in d2)
    y2.fill_(7)
    d2["dq"].fill_(7)
    assert both(ws.data_ptr(), need - 1)[1] == -8
    assert both(ws.data_ptr() + 4, ws.numel())[1] == -5
    torch.cuda.synchronize()
    assert (d2["dq"] == 7).all()


def test_graphs_replay_exactly():
    """A prompt, its gradients and token steps captured in two graphs: every replay equals the eager calls."""
    import torch

    import selective_state_space_35_amd as ssm

    x = make(b=2, L=600, H=4, G=2, Dk=64, Dv=64, seed=12)
    x2 = make(b=1, L=90, H=4, G=4, Dk=128, Dv=64, seed=13)
    say("linattn graphs")
    state = torch.empty_like(x["initial_state"])

    def work(z, with_token):
        y, last = fwd(z)
        d = bwd(z)
        out = [y, last, *[t for t in d.values() if t is not None]]
        if with_token:
            state.copy_(last)
            out.append(ssm.ssm_linattn_update(state, z["q"][:, 0].contiguous(), z["k"][:, 0].contiguous(),
                                              z["v"][:, 0].contiguous(), scale=z["scale"]))
            out.append(state)
        return out

    eager = [[t.clone() for t in work(x, True)], [t.clone() for t in work(x2, False)]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(x, True)
        work(x2, False)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for z, tok in ((x, True), (x2, False)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work(z, tok))
        graphs.append(g)
    for rep in range(4):
        for t in (*outs[0], *outs[1]):
            t.fill_(5)
        torch.cuda.synchronize()
        for g in graphs if rep % 2 else graphs[::-1]:
            g.replay()
        if rep == 2:
            fwd(x2)  # eager work beside the replays
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert all(torch.equal(s, t) for s, t in zip(a, b)), f"replay {rep}"


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: with decays of e^-1 a token, the first and the last tokens see only their
    neighbours, so short calls on those alone give the same values (up to e^-100, and the order of their chunks)."""
    import torch

    import selective_state_space_35_amd as ssm

    L, H, D, n = (1 << 18) + 77, 65, 128, 300
    say(f"linattn L={L} H={H} D={D}: {L * H * D / 2 ** 31:.2f} x 2^31 elements")
    if torch.cuda.mem_get_info()[0] < (80 << 30):
        pytest.skip("needs 80 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, dy = (torch.randn((1, L, H, D), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    A = torch.full((H,), -1.0, device="cuda")
    y, last = ssm.ssm_linattn_fwd(q, k, v, A=A)
    d = ssm.ssm_linattn_bwd(q, k, v, dy, A=A)
    torch.cuda.synchronize()
    for part, keep in ((slice(0, n), slice(0, n - 100)), (slice(L - n, L), slice(100, n))):
        t = [z[:, part].contiguous() for z in (q, k, v, dy)]
        y2, last2 = ssm.ssm_linattn_fwd(*t[:3], A=A)
        d2 = ssm.ssm_linattn_bwd(*t, A=A)
        torch.cuda.synchronize()
        for name, a, b in (("y", y, y2), *((m, d[m], d2[m]) for m in ("dq", "dk", "dv"))):
            a, b = a[:, part][:, keep].float(), b[:, keep].float()
            # two results of one definition: each within the documented bound, of which sums of about 1 / (1 - e^-1)
            # products make the magnitude; the state's and the mixing matrix's rounding to bf16 dominate
            e = (a - b).norm() / b.norm()
            assert e <= 4 * 2.0 ** -8, (name, part, float(e))
    e = (last - last2).norm() / last2.norm()
    assert e <= 1e-6, float(e)


def test_group_sums_of_more_elements_than_a_grid():
    """dq and dk of shared heads beyond 2^30 elements one at a time (Dk 33): equal batch rows, equal gradients."""
    import torch

    b, L, H, Dk = 512, 65536, 2, 33
    say(f"linattn bwd b={b} L={L} H={H} Dk={Dk}")
    if torch.cuda.mem_get_info()[0] < (80 << 30):
        pytest.skip("needs 80 GB of free memory")
    x = make(b=1, L=L, H=H, G=1, Dk=Dk, Dv=1, dtype="bf16", seed=5)
    d = bwd({n: t.expand(b, *t.shape[1:]).contiguous() if isinstance(t, torch.Tensor) else t for n, t in x.items()})
    torch.cuda.synchronize()
    for n in ("dq", "dk"):
        assert d[n].numel() > 1 << 30 and torch.isfinite(d[n][0]).all() and d[n][0].abs().max() > 0
        for i in range(0, b, 64):
            assert torch.equal(d[n][i:i + 64], d[n][:1].expand(64, L, 1, Dk)), (n, i)


def test_agrees_with_the_scalar_per_head_scan():
    """ssm_ssd_fwd is the case of one group: q = C, k = B, v = delta x, log decay delta A."""
    import torch

    import selective_state_space_35_amd as ssm
    import workloads
    from tests.parity import TOL

    w = workloads.SsdWorkload("linattn_ssd", b=2, L=300, H=3, N=64, gate=False, with_D=False, softplus=False)
    z = workloads.make_ssd_inputs(w, seed=2)
    z = {k: (t.cuda() if hasattr(t, "cuda") else t) for k, t in z.items()}
    delta = (z["delta"].float().abs() * 0.05).to(torch.bfloat16)
    say("linattn against the scalar-per-head scan")
    y, _ = ssm.ssm_ssd_fwd(z["x"], delta, z["A"], z["B"], z["C"])
    f = {"q": z["C"].float().view(2, 300, 1, 64), "k": z["B"].float().view(2, 300, 1, 64),
         "v": z["x"].float().view(2, 300, 3, 64) * delta.float()[..., None], "g": delta.float() * z["A"]}
    y2, _ = ssm.ssm_linattn_fwd(f["q"], f["k"], f["v"], g=f["g"], scale=1.0)
    torch.cuda.synchronize()
    e = ((y.float() - y2.reshape(y.shape)).abs() / (1 + y2.reshape(y.shape).abs())).max().item()
    assert e <= TOL["bf16"], e


def test_prompt_then_tokens_with_norms():
    """A layer in use: norm, linear attention over a padded batch of prompts, norm of each head, then tokens on
    the prompts' states; against the same layer over the whole sequences."""
    import torch

    import selective_state_space_35_amd as ssm

    b, L, T, H, D = 3, 150, 5, 4, 64
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    W = H * D
    lens = [150, 64, 1]
    u = n(b, L + T, W)
    wq, wk, wv = (n(W, W) * W ** -0.5 for _ in range(3))
    wg = n(W, H) * W ** -0.5
    lw, lb, hw, hb = 1 + 0.1 * n(W), 0.1 * n(W), 1 + 0.1 * n(H, D), 0.1 * n(H, D)

    def proj(z):
        z, _, _ = ssm.ssm_layernorm_fwd(z, lw, lb)
        f = lambda w: (z @ w).view(*z.shape[:-1], H, D).contiguous()  # noqa: E731
        return f(wq), f(wk), f(wv), -torch.nn.functional.softplus(z @ wg).contiguous()

    say("linattn prompt, tokens and norms")
    pad = torch.zeros(b, L, W, device="cuda")
    for i in range(b):
        pad[i, :lens[i]] = u[i, :lens[i]]
    q, k, v, g = proj(pad)
    _, state = ssm.ssm_linattn_fwd(q, k, v, g=g, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    got = []
    for t in range(T):
        tok = torch.stack([u[i, lens[i] + t] for i in range(b)])
        y = ssm.ssm_linattn_update(state, *(lambda q, k, v, g: (q, k, v, g))(*proj(tok)))
        got.append(ssm.ssm_layernorm_fwd(y, hw, hb)[0])
    got = torch.stack(got, 1)
    for i in range(b):
        q, k, v, g = proj(u[i:i + 1, :lens[i] + T].contiguous())
        y, _ = ssm.ssm_linattn_fwd(q, k, v, g=g)
        want = ssm.ssm_layernorm_fwd(y[:, lens[i]:].contiguous(), hw, hb)[0]
        # both sides in fp32; the norm divides by the spread of y, so errors are relative to the row
        assert ((got[i] - want[0]).abs().max() <= 2e-3), (got[i] - want[0]).abs().max()


def test_training_step_through_norms():
    """Gradients through norm, linear attention and the norm of each head, chained by hand, against float64
    automatic differentiation of the same layer."""
    import torch

    import selective_state_space_35_amd as ssm

    b, L, H, D = 2, 96, 3, 32
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v, g = n(b, L, H, D), n(b, L, H, D), n(b, L, H, D), -0.2 * n(b, L, H).abs()
    w, c = 1 + 0.1 * n(H, D), 0.1 * n(H, D)
    dout = n(b, L, H, D)
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, w, c)]
    Q, K, V, Gt, Wt, Ct = leaves
    qn = torch.nn.functional.layer_norm(Q, (D,))
    cum = Gt.cumsum(1)
    mask = torch.tril(torch.ones(L, L, dtype=torch.bool))[None, :, :, None]
    diff = (cum[:, :, None] - cum[:, None]).masked_fill(~mask, -math.inf)
    p = torch.einsum("bthd,bshd->btsh", qn, K) * D ** -0.5 * diff.exp()
    y = torch.einsum("btsh,bshd->bthd", p, V)
    out = torch.nn.functional.layer_norm(y, (D,)) * Wt + Ct
    (out * dout).sum().backward()
    want = [t.grad for t in leaves]
    say("linattn training step")
    q, k, v, g, w, c, dout = (t.cuda() for t in (q, k, v, g, w, c, dout))
    qn, m1, r1 = ssm.ssm_layernorm_fwd(q)
    y, _ = ssm.ssm_linattn_fwd(qn, k, v, g=g)
    _, m2, r2 = ssm.ssm_layernorm_fwd(y, w, c)
    dn = ssm.ssm_layernorm_bwd(y, dout, m2, r2, w)
    d = ssm.ssm_linattn_bwd(qn, k, v, dn["dx"], g=g)
    dq = ssm.ssm_layernorm_bwd(q, d["dq"], m1, r1, param_grads=False)["dx"]
    for name, got, ref in zip(("q", "k", "v", "g", "w", "b"), (dq, d["dk"], d["dv"], d["dg"], dn["dweight"], dn["dbias"]), want):
        rel = ((got.double().cpu() - ref).norm() / ref.norm()).item()
        print(f"[linattn] training step d{name}: relative error {rel:.2e}", flush=True)
        # fp32 throughout: some hundreds of roundings of 2^-24, relative to sums that partly cancel
        assert rel <= 2e-5, (name, rel)
