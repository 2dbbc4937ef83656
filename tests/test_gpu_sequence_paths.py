"""The sequence operators where a rule on sizes chooses another path, for torch's automatic
differentiation, and together in the example model."""
import os
import sys

import numpy as np
import pytest
import torch

import sequence_ref as ref
import stream_compaction_amd as sc
from stream_compaction_amd import autograd as ops
from test_gpu_sequence import TYPES, act, agree, gen, host, par, scan_inputs

pytestmark = pytest.mark.gpu


# many sequences of few channels: two tiles per workgroup in the gradient, the second one
# whole, in part or missing; with a state and a group left over
@pytest.mark.parametrize("case", [
    (128, 20, 32, 16, 1, "bf16", None, "gate soft bias D init"),
    (130, 35, 41, 13, 1, "f32", "ragged", "soft bias D"),
    (64, 17, 80, 16, 2, "f16", "ragged", "gate soft bias D init"),
], ids=["whole", "odd", "groups"])
def test_scan_grad_two_tiles(case):
    case = list(case)
    if case[6] == "ragged":
        case[6] = [(7 * i) % (case[1] + 2) for i in range(case[0])]
    k, w, dy, dfinal = scan_inputs(tuple(case), 200, grads=True)
    y, state, starts = sc.selective_scan(keep_starts=True, **k)
    k.pop("initial_state", None)
    got = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    again = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    want = ref.scan(**w)
    agree(y, want["y"], case[5], "y")
    for name, v in got.items():
        if v is not None:
            agree(v, want[name], case[5] if v.dtype != torch.float32 else "f32", name)
            assert torch.equal(v, again[name])


# few channels over a length that is cut into chunks: sequences that end inside a chunk, at its
# border, before it, and nowhere
@pytest.mark.parametrize("case", [
    (1, 1500, 20, 16, 1, "bf16", None, "gate soft bias D init"),
    (3, 1300, 18, 13, 1, "f32", [1300, 417, 0], "soft bias D init"),
    (2, 1024, 34, 16, 2, "f16", [512, 1], "gate soft bias D"),
    (1, 700, 6, 33, 1, "bf16", None, "gate soft bias D init"),
    (2, 4099, 5, 4, 1, "f32", [4099, 2049], "gate D init"),
], ids=["whole", "ragged", "border", "states", "long"])
def test_scan_in_chunks(case):
    k, w, dy, dfinal = scan_inputs(case, 290, grads=True)
    y, state, starts = sc.selective_scan(keep_starts=True, **k)
    y2, state2 = sc.selective_scan(**k)
    init = k.pop("initial_state", None)
    got = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    again = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    want = ref.scan(**w)
    assert torch.equal(y, y2) and torch.equal(state, state2)
    agree(y, want["y"], case[5], "y")
    agree(state, want["state"], "f32", "state")
    for name, v in got.items():
        if v is not None:
            agree(v, want[name], case[5] if v.dtype != torch.float32 else "f32", name)
            assert torch.equal(v, again[name])
    # the whole scan in one piece gives the same but for rounding, and so do two halves in turn
    half = case[1] // 2
    if case[6] is None:
        part = {n: k[n][:, :half] for n in ("x", "dt", "B", "C") + (("z",) if "z" in k else ())}
        rest = {n: k[n][:, half:] for n in part}
        a, mid = sc.selective_scan(**{**k, **part}, initial_state=init)
        b, end = sc.selective_scan(**{**k, **rest}, initial_state=mid)
        cut = lambda v, s: ref.V(v.val[:, s], v.mag[:, s], v.err[:, s])  # noqa: E731
        agree(a, cut(want["y"], slice(None, half)), case[5], "first half")
        agree(b, cut(want["y"], slice(half, None)), case[5], "second half")
        agree(end, want["state"], "f32", "state after both")


def test_conv_long_runs():
    # enough lanes for the longest runs; in two parts the runs are shorter, the sums the same
    x = torch.randn(1, 16391, 4096, generator=gen(210)).bfloat16().cuda()
    w, bias = par(gen(211), (4096, 4), 0.5)[0], par(gen(212), (4096,))[0]
    y, state = sc.causal_conv(x, w, bias)
    cut = 5003
    y1, mid = sc.causal_conv(x[:, :cut], w, bias)
    y2, last = sc.causal_conv(x[:, cut:], w, bias, initial_state=mid)
    assert torch.equal(y, torch.cat([y1, y2], 1)) and torch.equal(state, last)
    dy = torch.randn(1, 16391, 4096, generator=gen(213)).bfloat16().cuda()
    g = sc.causal_conv_grad(dy, x, w, bias)
    g2 = sc.causal_conv_grad(dy[:, cut:], x[:, cut:], w, bias, initial_state=mid)
    g1 = sc.causal_conv_grad(dy[:, :cut], x[:, :cut], w, bias, dfinal=g2["dstate"])
    assert torch.equal(g["dx"][:, cut:], g2["dx"])
    assert torch.equal(g["dx"][:, :cut - 3], g1["dx"][:, :-3])


def test_scan_step_many_sequences():
    # two sequences a lane, and the one left over; fewer take another path
    d, n = 4096, 16
    for b in (128, 131):
        r = gen(220 + b)
        state = par(r, (b, d, n))[0]
        x, dt, z = (act(r, (b, d), "bf16")[0] for _ in range(3))
        B, C = (act(r, (b, 1, n), "bf16")[0] for _ in range(2))
        A, D, bias = -torch.rand((d, n), generator=r).cuda(), par(r, (d,))[0], par(r, (d,), 0.5, -3)[0]
        new = torch.empty_like(state)
        y = sc.selective_scan_step(state, x, dt, A, B, C, D, z, bias, softplus=True, new_state=new)
        for i in (0, 1, b // 2, b - 2, b - 1):
            s = slice(i, i + 1)
            one = torch.empty_like(state[s])
            v = sc.selective_scan_step(state[s], x[s], dt[s], A, B[s], C[s], D, z[s], bias,
                                       softplus=True, new_state=one)
            assert torch.equal(v, y[s]) and torch.equal(one, new[s])


@pytest.mark.parametrize("tokens,rows,d", [(16384, 700, 8), (16385, 700, 8), (16384, 700, 133), (300, 131072, 8),
                                           (300, 131073, 8), (1024, 65537, 16), (2, 1 << 24, 2)])
def test_embedding_grad_paths(tokens, rows, d):
    r = gen(230)
    dout, dr = act(r, (tokens, d), "f32")
    ids = torch.randint(-1, rows + 1, (tokens,), generator=r)
    ids[::3] = rows - 1
    got = sc.embedding_grad(dout, ids.cuda(), rows)
    idn = ids.numpy()
    live = (idn >= 0) & (idn < rows)
    used, where = np.unique(idn[live], return_inverse=True)
    depth = 34 + int(np.bincount(where).max()) // 8 if live.any() else 1
    want = ref.embedding_grad(dr[live], where, len(used), 1.0, depth)
    agree(got[torch.from_numpy(used).cuda()], want, "f32", "rows with tokens")
    got[torch.from_numpy(used).cuda()] = 0
    assert not bool(got.any())


def test_embedding_past_the_caches():
    # an output that is stored past the caches: with scale 1 a copy of the rows
    r = gen(235)
    table = torch.randn(300, 2048, generator=r).bfloat16().cuda()
    ids = torch.randint(-1, 301, (8200,), generator=r).cuda()
    live = (ids >= 0) & (ids < 300)
    want = torch.where(live[:, None], table[ids.clamp(0, 299)], torch.zeros((), dtype=torch.bfloat16,
                                                                           device="cuda"))
    assert torch.equal(sc.embedding(table, ids), want)


def test_explicit_stream():
    case = (2, 90, 48, 16, 1, "bf16", None, "gate soft bias D init")
    k, _, dy, dfinal = scan_inputs(case, 240, grads=True)
    want = sc.selective_scan(keep_starts=True, **k)
    ids = torch.arange(96, device="cuda") % 7
    wide = torch.randn(96, 48, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sc.selective_scan(keep_starts=True, stream=s, **k)
    k.pop("initial_state")
    g = sc.selective_scan_grad(dy, starts=got[2], dfinal=dfinal, stream=s, **k)
    e = sc.embedding_grad(wide, ids, 7, stream=s)
    s.synchronize()
    h = sc.selective_scan_grad(dy, starts=want[2], dfinal=dfinal, **k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(g[n], h[n]) for n in g)
    assert torch.equal(e, sc.embedding_grad(wide, ids, 7))


# ---- automatic differentiation ----
def leaf(t):
    return t.detach().clone().requires_grad_(True)


def test_autograd_is_the_gradient():
    case = (2, 50, 24, 16, 2, "f32", [50, 31], "gate soft bias D init")
    k, _, dy, dfinal = scan_inputs(case, 250, grads=True)
    for name in ("x", "dt", "B", "C", "z"):
        k[name] = torch.nan_to_num(k[name], 0.0, 0.0, 0.0)
    dy = torch.nan_to_num(dy, 0.0, 0.0, 0.0)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial_state")
    leaves = {n: leaf(k[n]) for n in names}
    y, state = ops.selective_scan(**leaves, softplus=True, lengths=k["lengths"])
    torch.autograd.backward([y, state], [dy, dfinal])
    _, _, starts = sc.selective_scan(keep_starts=True, **k)
    k.pop("initial_state")
    g = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    for n in names:
        key = "dstate" if n == "initial_state" else "d" + n if n != "dt_bias" else "ddt_bias"
        assert torch.equal(leaves[n].grad, g[key]), n
    # the state alone, and a sum's expanded gradient
    more = {n: leaves[n] for n in names}
    _, state = ops.selective_scan(**more, softplus=True)
    a, = torch.autograd.grad(state.sum(), leaves["x"])
    y, _ = ops.selective_scan(**more, softplus=True)
    b, = torch.autograd.grad(y.sum(), leaves["x"])
    y, _ = ops.selective_scan(**more, softplus=True)
    c, = torch.autograd.grad(y, leaves["x"], torch.ones_like(y))
    assert bool(torch.isfinite(a).all()) and torch.equal(b, c)


def test_autograd_conv_and_embedding():
    r = gen(260)
    x, w, bias, init = (leaf(t) for t in (act(r, (2, 30, 20), "f32")[0], par(r, (20, 4))[0],
                                          par(r, (20,))[0], act(r, (2, 3, 20), "f32")[0]))
    y, state = ops.causal_conv(x, w, bias, init)
    dy, df = torch.randn_like(y), torch.randn_like(state)
    torch.autograd.backward([y, state], [dy, df])
    g = sc.causal_conv_grad(dy, x.detach(), w.detach(), bias.detach(), init.detach(), dfinal=df)
    for t, n in ((x, "dx"), (w, "dweight"), (bias, "dbias"), (init, "dstate")):
        assert torch.equal(t.grad, g[n])
    table = leaf(act(r, (50, 20), "f32")[0])
    ids = torch.randint(-1, 50, (3, 11), generator=r).cuda()
    out = ops.embedding(table, ids, 2.0)
    dout = torch.randn_like(out)
    out.backward(dout)
    assert torch.equal(table.grad, sc.embedding_grad(dout, ids, 50, 2.0))


def test_autograd_broadcast_inputs():
    # one step per channel and one B for the batch, expanded: their gradients are sums
    r = gen(270)
    b, l, d, n = 3, 40, 18, 8
    x = act(r, (b, l, d), "f32")[0]
    A = -torch.rand((d, n), generator=r).cuda()
    C = act(r, (b, l, 1, n), "f32")[0]
    dt, B = leaf(torch.rand((d,), generator=r).cuda() * 0.1), leaf(act(r, (1, l, 1, n), "f32")[0])
    y, _ = ops.selective_scan(x, dt.expand(b, l, d), A, B.expand(b, l, 1, n), C)
    dy = torch.randn(y.shape, generator=r).cuda()
    y.backward(dy)
    full_dt, full_B = dt.detach().expand(b, l, d).contiguous(), B.detach().expand(b, l, 1, n).contiguous()
    _, _, starts = sc.selective_scan(x, full_dt, A, full_B, C, keep_starts=True)
    g = sc.selective_scan_grad(dy, x, full_dt, A, full_B, C, starts)
    assert torch.allclose(dt.grad, g["ddt"].sum((0, 1)), rtol=1e-5, atol=1e-5)
    assert torch.allclose(B.grad, g["dB"].sum(0, keepdim=True), rtol=1e-5, atol=1e-5)


def test_scan_gradient_against_differences():
    # the kernels' gradient along a direction against the float64 oracle's slope along it
    case = (2, 33, 10, 5, 1, "f32", [33, 20], "gate soft bias D init")
    k, w, dy, dfinal = scan_inputs(case, 280, grads=True)
    _, _, starts = sc.selective_scan(keep_starts=True, **k)
    k.pop("initial_state")
    got = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    want = ref.scan(**w)
    rng = np.random.default_rng(0)
    live = np.arange(33)[None, :] < np.array([33, 20])[:, None]

    def loss(moved):
        o = ref.scan(**{**w, **moved, "dy": None, "dfinal": None})
        return float((np.where(live[..., None], w["dy"], 0) * o["y"].val).sum() +
                     (w["dfinal"] * o["state"].val).sum())

    step = 1e-5
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"),
                      ("z", "dz"), ("dt_bias", "ddt_bias"), ("initial", "dstate")):
        v = rng.standard_normal(w[name].shape)
        up, down = loss({name: w[name] + step * v}), loss({name: w[name] - step * v})
        slope = (up - down) / (2 * step)
        along = float((host(got[key]) * v).sum())
        # the gradient's own bound along v, and differences of order step^2 on slopes of order 1
        room = float(((want[key].err + 2.0 ** -24 * np.abs(want[key].val)) * np.abs(v)).sum())
        room += 1e-8 * float((np.abs(want[key].mag) * np.abs(v)).sum())
        assert abs(slope - along) <= room, (name, slope, along, room)


def test_backward_in_a_graph():
    # forward and backward captured together, replayed on new inputs
    r = gen(290)
    rows, d, n, shape = 61, 32, 16, (2, 45)
    make = lambda: [t.clone() for t in (  # noqa: E731
        table, w, bias, A, D)]
    table, w, bias = act(r, (rows, d), "bf16")[0], par(r, (d, 4))[0], par(r, (d,))[0]
    A, D = -torch.rand((d, n), generator=r).cuda(), par(r, (d,))[0]
    dt, B, C = (act(r, s, "bf16", 0.3)[0] for s in (shape + (d,), shape + (1, n), shape + (1, n)))
    ids = torch.randint(-1, rows, shape, generator=r).cuda()
    dy = act(r, shape + (d,), "bf16")[0]

    def work(leaves):
        t, w, bias, A, D = leaves
        c, _ = ops.causal_conv(ops.embedding(t, ids, 2.0), w, bias)
        y, _ = ops.selective_scan(c, dt, A, B, C, D, softplus=True)
        return [y] + list(torch.autograd.grad(y, leaves, dy))

    captured = [t.requires_grad_(True) for t in make()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(captured)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(captured)
    eager = [t.requires_grad_(True) for t in make()]
    for i in range(3):
        ids.copy_(torch.randint(-1, rows, shape, generator=r))
        dy.copy_(torch.randn(dy.shape, generator=r))
        want = [t.detach().clone() for t in work(eager)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"replay {i}, output {j}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_example_model_learns_and_steps_agree(dtype):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import state_space_lm
    r = state_space_lm.run(steps=80, dtype=dtype)
    assert r["last"] < 0.1 * r["first"] and r["right"] > 0.9
    # steps and whole sequences round at different places: some steps of the type, a few layers
    assert r["off"] <= 64 * float(torch.finfo(TYPES[dtype]).eps) * r["span"]
