"""The gated scan on the GPU against the float64 oracle of ``gated_ref`` (whose bounds count float32
roundings), over the sizes, masks, strides and types where the kernels can go wrong; its gradient and
step against the operator they belong to."""
import math

import numpy as np
import pytest
import torch

import gated_ref as ref
import sequence_ref
import stream_compaction_amd as sc
from stream_compaction_amd import autograd as ops
from test_gpu_sequence import TYPES, act, agree, gen, host, par, poison, strided

pytestmark = pytest.mark.gpu

# batch, length, channels, type, lengths (None: all), options
CASES = [
    (1, 1, 1, "f32", None, ""),
    (1, 1, 64, "bf16", None, "rate in gate init"),
    (2, 0, 5, "f32", None, "rate init"),
    (1, 15, 2, "bf16", None, "rate in"),
    (2, 16, 129, "f32", None, "in gate init"),
    (1, 17, 128, "f16", None, "rate gate init"),
    (1, 63, 130, "bf16", None, "rate in gate init"),
    (2, 64, 33, "f32", None, "rate in init"),
    (3, 65, 7, "f16", [65, 0, 1], "rate in gate init"),
    (1, 127, 256, "bf16", None, ""),
    (2, 128, 24, "bf16", [128, 37], "rate in gate init"),
    (2, 129, 31, "f32", [129, 128], "rate in gate init"),
    (3, 200, 300, "bf16", [0, 200, 1], "rate gate init"),
    (1, 257, 3, "f32", None, "rate in"),
    (2, 513, 66, "f16", [513, 512], "in init"),
    (1, 1100, 34, "bf16", None, "rate in gate init"),
    (1, 2300, 1, "f32", None, "rate in init"),
    (1, 4200, 20, "f32", None, "rate in gate init"),
    (2, 4500, 9, "bf16", [4500, 2049], "gate init"),
    (5, 300, 19, "f32", [300, -3, 0, 900, 129], "rate in init"),
    (64, 70, 130, "bf16", None, "rate in"),
]
IDS = [f"{c[:4]}".replace(" ", "") for c in CASES]


def inputs(case, seed, grads=False):
    b, l, d, dt, lengths, opts = case
    r = gen(seed)
    k, w = {}, {"rate": None, "input_gate": None, "z": None, "initial": None}
    k["x"], w["x"] = act(r, (b, l, d), dt)
    # (without a rate the gate itself has to hold a state for long)
    shift = 0.0 if "rate" in opts else 3.0
    f = (torch.randn((b, l, d), generator=r) + shift).to(TYPES[dt])
    k["forget"], w["forget"] = f.cuda(), f.double().numpy()
    if "rate" in opts:
        # from holding over thousands of tokens to hardly at all
        rate = torch.exp(torch.rand(d, generator=r) * math.log(1e4)) * 5e-4
        k["rate"], w["rate"] = rate.cuda(), rate.double().numpy()
    if "in" in opts.split():
        k["input_gate"], w["input_gate"] = act(r, (b, l, d), dt)
    if "gate" in opts:
        k["z"], w["z"] = act(r, (b, l, d), dt)
    if "init" in opts:
        k["initial_state"], w["initial"] = par(r, (b, d))
    if lengths is not None:
        for name in ("x", "forget", "input_gate", "z"):
            if name in k:
                poison(k[name], lengths)
        k["lengths"] = torch.tensor(lengths, dtype=torch.int32).cuda()
        w["lengths"] = np.minimum(np.array(lengths), l)
    if grads:
        dy, w["dy"] = act(r, (b, l, d), dt)
        dfinal, w["dfinal"] = par(r, (b, d))
        return k, w, poison(dy, lengths), dfinal
    return k, w


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_scan(case):
    k, w = inputs(case, 10)
    y, state = sc.gated_scan(**k)
    want = ref.gated(**w)
    agree(y, want["y"], case[3], "y")
    agree(state, want["state"], "f32", "state")
    y2, state2 = sc.gated_scan(**k)
    assert torch.equal(y, y2) and torch.equal(state, state2)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_grad(case):
    k, w, dy, dfinal = inputs(case, 20, grads=True)
    y, state, starts = sc.gated_scan(keep_starts=True, **k)
    k.pop("initial_state", None)
    got = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    again = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    want = ref.gated(**w)
    agree(y, want["y"], case[3], "y")
    for name in ("dx", "dforget", "dinput_gate", "dz"):
        if got[name] is not None:
            agree(got[name], want[name], case[3], name)
    for name in ("drate", "dstate"):
        if got[name] is not None:
            agree(got[name], want[name], "f32", name)
    for name, arg in (("drate", "rate"), ("dinput_gate", "input_gate"), ("dz", "z")):
        assert (got[name] is None) == (arg not in k)
    for name, v in got.items():
        assert v is None or torch.equal(v, again[name]), f"{name} differs from call to call"
    no_final = sc.gated_scan_grad(dy, starts=starts, **k)
    w["dfinal"] = None
    agree(no_final["dstate"], ref.gated(**w)["dstate"], "f32", "dstate without dfinal")


@pytest.mark.parametrize("how", ["halves", "shifted", "time_major"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("channels", [48, 47])
def test_strides(how, dt, channels):
    case = (2, 330, channels, dt, [330, 177], "rate in gate init")
    k, _, dy, dfinal = inputs(case, 30, grads=True)
    y, state, starts = sc.gated_scan(keep_starts=True, **k)
    acts = ("x", "forget", "input_gate", "z")
    s = {n: strided(v, how) if n in acts else v for n, v in k.items()}
    y2, state2, starts2 = sc.gated_scan(keep_starts=True, **s)
    assert torch.equal(y, y2) and torch.equal(state, state2)
    k.pop("initial_state"), s.pop("initial_state")
    g1 = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    g2 = sc.gated_scan_grad(strided(dy, how), starts=starts2, dfinal=dfinal, **s)
    for name in g1:
        assert torch.equal(g1[name], g2[name]), name
    tok = {n: v[:, 5] if n in acts else v for n, v in k.items() if n != "lengths"}
    tok2 = {n: v[:, 5] if n in acts else v for n, v in s.items() if n != "lengths"}
    st, st2 = state.clone(), state.clone()
    assert torch.equal(sc.gated_scan_step(st, **tok), sc.gated_scan_step(st2, **tok2))
    assert torch.equal(st, st2)


@pytest.mark.parametrize("channels,dt", [(4096, "bf16"), (4090, "f16"), (8190, "f32"), (8191, "bf16"), (3968, "bf16")])
def test_wide_rows(channels, dt):
    # many channels a row; each is its own, with the same bits as in a row of a few (an odd row
    # goes by another kernel, whose sums and products the compiler may join otherwise)
    test_scan((2, 300, channels, dt, [300, 190], "rate in gate init"))
    test_grad((2, 300, channels, dt, [300, 190], "rate in gate init"))
    if channels % 2:
        return
    k, _, dy, dfinal = inputs((2, 300, channels, dt, [300, 190], "rate in gate init"), 35, grads=True)
    y, state, starts = sc.gated_scan(keep_starts=True, **k)
    initial = k.pop("initial_state")
    g = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    starts = starts.view(2, -1, channels)
    for lo, hi in ((0, 130), (900, 1156), (channels - 390, channels)):
        part = {n: v if n == "lengths" else v[..., lo:hi].contiguous() for n, v in k.items()}
        y2, state2, starts2 = sc.gated_scan(keep_starts=True, initial_state=initial[:, lo:hi].contiguous(), **part)
        assert torch.equal(y[..., lo:hi], y2) and torch.equal(state[:, lo:hi], state2), (lo, hi)
        for i, blocks in ((0, 5), (1, 3)):                   # (none is written for blocks without a token)
            assert torch.equal(starts[i, :blocks, lo:hi], starts2.view(2, 5, -1)[i, :blocks]), (lo, hi)
        g2 = sc.gated_scan_grad(dy[..., lo:hi].contiguous(), starts=starts2, dfinal=dfinal[:, lo:hi].contiguous(), **part)
        for name in g:
            assert torch.equal(g[name][..., lo:hi], g2[name]), (lo, hi, name)


def test_broadcast_strides():
    # one token of the gate and one batch of z, repeated with stride 0; a row of one value
    k, _ = inputs((3, 170, 20, "f32", None, "rate in gate"), 40)
    k["forget"] = k["forget"][:, :1].expand(3, 170, 20)
    k["z"] = k["z"][:1].expand(3, -1, -1)
    y, state = sc.gated_scan(**k)
    y2, state2 = sc.gated_scan(**{n: v.contiguous() for n, v in k.items()})
    assert torch.equal(y, y2) and torch.equal(state, state2)


def cut_of(v, where):
    return sequence_ref.V(v.val[:, where], v.mag[:, where], v.err[:, where])


@pytest.mark.parametrize("opts", ["rate in gate init", "init"])
def test_in_parts_and_steps(opts):
    # a sequence scanned in two parts, then token by token, is the whole one's
    k, w = inputs((2, 360, 37, "f32", None, opts), 50)
    want = ref.gated(**w)
    acts = [n for n in ("x", "forget", "input_gate", "z") if n in k]
    init = k.pop("initial_state")
    more = {n: v for n, v in k.items() if n not in acts}
    y1, a = sc.gated_scan(**{n: k[n][:, :131] for n in acts}, **more, initial_state=init)
    y2, mid = sc.gated_scan(**{n: k[n][:, 131:330] for n in acts}, **more, initial_state=a)
    agree(torch.cat([y1, y2], 1), cut_of(want["y"], slice(0, 330)), "f32", "parts")
    ys = [sc.gated_scan_step(mid, **{n: k[n][:, t] for n in acts}, **more) for t in range(330, 360)]
    agree(torch.stack(ys, 1), cut_of(want["y"], slice(330, 360)), "f32", "steps")
    agree(mid, want["state"], "f32", "state")


@pytest.mark.parametrize("b,d,dt", [(1, 1, "f32"), (3, 17, "bf16"), (2, 40, "f16"), (130, 64, "bf16"),
                                    (1, 4096, "bf16"), (5, 333, "f32"), (64, 1026, "f16")])
@pytest.mark.parametrize("opts", ["", "rate in gate", "rate", "in gate"])
def test_step(b, d, dt, opts):
    k, w = inputs((b, 1, d, dt, None, opts + " init"), 60)
    want = ref.gated(**w)
    state = k.pop("initial_state")
    tok = {n: v[:, 0] if v.dim() == 3 else v for n, v in k.items()}
    before, fresh = state.clone(), torch.empty_like(state)
    y = sc.gated_scan_step(state, new_state=fresh, **tok)
    assert torch.equal(state, before)
    agree(y, cut_of(want["y"], 0), dt, "y")
    agree(fresh, want["state"], "f32", "state")
    y2 = sc.gated_scan_step(state, **tok)
    assert torch.equal(y, y2) and torch.equal(state, fresh)


def test_far_offsets():
    # strides that pass 2^31 elements and 2^32 bytes
    step = (1 << 30) + 8
    big = torch.zeros(2 * step + 64, dtype=torch.bfloat16, device="cuda")
    r = gen(100)
    x0 = act(r, (1, 3, 16), "bf16")[0]
    far = big.as_strided((1, 3, 16), (3 * step, step, 1))
    far.copy_(x0)
    rate = torch.rand(16, generator=r).cuda()
    y1, s1, k1 = sc.gated_scan(far, far, rate, far, far, keep_starts=True)
    y0, s0, k0 = sc.gated_scan(x0, x0, rate, x0, x0, keep_starts=True)
    assert torch.equal(y1, y0) and torch.equal(s1, s0)
    g1 = sc.gated_scan_grad(far, far, far, k1, rate, far, far)
    g0 = sc.gated_scan_grad(x0, x0, x0, k0, rate, x0, x0)
    assert all(torch.equal(g1[n], g0[n]) for n in g0)
    del big, far
    torch.cuda.empty_cache()


@pytest.mark.parametrize("opts", ["rate in init", "gate"])
def test_past_the_caches(opts):
    # 34 MB an output, loaded and stored past the caches: with states kept and without, against some channels alone
    k, w, dy, dfinal = inputs((2, 2100, 4096, "bf16", [2100, 1300], opts), 105, grads=True)
    y, state, starts = sc.gated_scan(keep_starts=True, **k)
    y2, state2 = sc.gated_scan(**k)
    k.pop("initial_state", None)
    g = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    for lo, hi in ((0, 20), (2040, 2060), (4076, 4096)):
        want = ref.gated(**{n: v if n == "lengths" or v is None else v[..., lo:hi] for n, v in w.items()})
        for what, got in (("y", y), ("y", y2), ("dx", g["dx"]), ("dforget", g["dforget"]),
                          ("dinput_gate", g["dinput_gate"]), ("dz", g["dz"])):
            if got is not None:
                agree(got[..., lo:hi], want[what], "bf16", what)
        for what, got in (("state", state), ("state", state2), ("drate", g["drate"]), ("dstate", g["dstate"])):
            if got is not None:
                agree(got[..., lo:hi], want[what], "f32", what)


def test_far_outputs():
    # an output that passes 2^32 bytes; the sequence's end against the end alone
    l, d = 40001, 54001
    x = torch.randn(1, l, 1, device="cuda").bfloat16().expand(1, l, d).contiguous()
    f = torch.full((1, 1, 1), 2.0, dtype=torch.bfloat16, device="cuda").expand(1, 1, d).contiguous()
    y, state = sc.gated_scan(x, f.expand(1, l, d))
    assert torch.equal(y[..., 0], y[..., d - 1]) and torch.equal(state[:, 0], state[:, d - 1])
    y1, state1 = sc.gated_scan(x[..., :1].contiguous(), f[..., :1].expand(1, l, 1))
    assert torch.equal(y[:, ::997, 5], y1[:, ::997, 0]) and torch.equal(state[:, 77], state1[:, 0])
    del x, y
    torch.cuda.empty_cache()


def test_another_stream_and_two_at_once():
    case = (2, 900, 48, "bf16", [900, 611], "rate in gate init")
    k, _, dy, dfinal = inputs(case, 110, grads=True)
    y, state, starts = sc.gated_scan(keep_starts=True, **k)
    grads = {n: v for n, v in k.items() if n != "initial_state"}
    g = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **grads)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 3]):
            y2, state2, starts2 = sc.gated_scan(keep_starts=True, **k)
            outs.append((y2, state2, sc.gated_scan_grad(dy, starts=starts2, dfinal=dfinal, **grads)))
    torch.cuda.synchronize()
    for y2, state2, g2 in outs:
        assert torch.equal(y, y2) and torch.equal(state, state2)
        assert all(torch.equal(g[n], g2[n]) for n in g)
    # a stream that is given, with the caller's own scratch
    need = 1 << 22
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    y3, state3 = sc.gated_scan(scratch=scratch, stream=streams[0], **k)
    streams[0].synchronize()
    assert torch.equal(y, y3) and torch.equal(state, state3)


def test_graph_replays():
    # two graphs of the whole path, each replayed on new inputs with eager work between
    case = (2, 700, 130, "bf16", [700, 400], "rate in gate init")
    k, _, dy, dfinal = inputs(case, 120, grads=True)
    acts = ("x", "forget", "input_gate", "z")
    for n in acts:
        k[n] = torch.nan_to_num(k[n], posinf=0.0)
    dy = torch.nan_to_num(dy, posinf=0.0)
    init = k.pop("initial_state")

    def work():
        y, state, starts = sc.gated_scan(keep_starts=True, initial_state=init, **k)
        g = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
        st = state.clone()
        tok = {n: v[:, 3] if n in acts else v for n, v in k.items() if n != "lengths"}
        v = sc.gated_scan_step(st, **tok)
        return [y, state, v, st, *g.values()]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = work()
        graphs.append((graph, outs))
    r = gen(121)
    for i in range(4):
        for n in acts:
            k[n].copy_(torch.randn(k[n].shape, generator=r))
        want = [t.clone() for t in work()]
        torch.cuda.synchronize()
        for graph, outs in graphs:
            graph.replay()
            torch.cuda.synchronize()
            for j, (a, b) in enumerate(zip(outs, want)):
                assert torch.equal(a, b), f"replay {i}, output {j}"


@pytest.mark.parametrize("opts", ["rate in gate init", "in", ""])
def test_autograd(opts):
    k, w, dy, dfinal = inputs((2, 150, 20, "f32", [150, 61], opts), 130, grads=True)
    leaves = {n: v.clone().requires_grad_() for n, v in k.items() if n != "lengths"}
    y, state = ops.gated_scan(**leaves, lengths=k["lengths"])
    torch.autograd.backward([y, state], [dy, dfinal])
    want = ref.gated(**w)
    names = {"x": "dx", "forget": "dforget", "rate": "drate", "input_gate": "dinput_gate", "z": "dz",
             "initial_state": "dstate"}
    for n, v in leaves.items():
        agree(v.grad, want[names[n]], "f32", n)
    # gradients of the state alone, and of a sum (an expanded single value)
    for v in leaves.values():
        v.grad = None
    y, state = ops.gated_scan(**leaves, lengths=k["lengths"])
    y.sum().backward()
    w2 = {**w, "dy": np.ones_like(w["dy"]), "dfinal": None}
    agree(leaves["x"].grad, ref.gated(**w2)["dx"], "f32", "dx of a sum")


def test_differences():
    # the gradient against differences of the operator itself, in float32: a step of 2^-6 moves the
    # loss by far more than its rounding (2^-24 of a sum of 30 x 7 terms of about 1, over 2^-5)
    k, _, dy, _ = inputs((1, 30, 7, "f32", None, "rate in gate init"), 140, grads=True)
    k["rate"] = k["rate"].clamp(0.05, 2.0)
    leaves = {n: v.clone().requires_grad_() for n, v in k.items()}
    (ops.gated_scan(**leaves)[0] * dy).sum().backward()
    r = gen(141)
    for name in leaves:
        way = torch.randn(k[name].shape, generator=r).cuda()
        way /= way.norm()
        step = 2.0 ** -6
        up = (sc.gated_scan(**{**k, name: k[name] + step * way})[0].double() * dy).sum()
        low = (sc.gated_scan(**{**k, name: k[name] - step * way})[0].double() * dy).sum()
        slope = float((up - low) / (2 * step))
        want = float((leaves[name].grad.double() * way).sum())
        scale = float(leaves[name].grad.norm())
        # (third derivatives are of the gradient's size: step^2 / 6 of it, and up to 30 times that
        # through rates as small as 0.05)
        assert abs(slope - want) < 2e-3 * scale + 1e-4, name


def test_infinities_and_rates_at_their_ends():
    # what a channel does stays in it; a rate of 0 or less holds the state, an infinite one forgets
    b, l, d = 1, 700, 12
    r = gen(150)
    x, f, i = (act(r, (b, l, d), "f32")[0] for _ in range(3))
    rate = torch.rand(d, generator=r).cuda()
    clean = sc.gated_scan(x, f, rate, i)
    rate2, x2, f2 = rate.clone(), x.clone(), f.clone()
    rate2[1], rate2[2], rate2[3] = 0.0, -3.0, float("inf")
    x2[0, 200, 5] = float("inf")
    x2[0, 300, 7] = float("nan")
    f2[0, 100, 8], f2[0, 400, 9] = float("-inf"), float("inf")
    init = torch.randn((b, d), generator=r).cuda()
    y, state, starts = sc.gated_scan(x2, f2, rate2, i, initial_state=init, keep_starts=True)
    ref_y, ref_s = sc.gated_scan(x, f, rate, i, initial_state=init)
    same = [0, 4, 6, 10, 11]
    assert torch.equal(y[..., same], ref_y[..., same]) and torch.equal(state[:, same], ref_s[:, same])
    for c in (1, 2):
        assert bool((y[0, :, c] == init[0, c]).all()) and float(state[0, c]) == float(init[0, c])
    v = torch.sigmoid(i[0, :, 3].double()) * x2[0, :, 3].double()
    assert torch.allclose(y[0, :, 3].double(), v, rtol=1e-6, atol=1e-7)
    assert bool(torch.isfinite(state[:, [0, 1, 2, 3, 4, 6, 8, 9, 10, 11]]).all())
    assert bool(torch.isfinite(y[0, :200, 5]).all()) and bool(torch.isinf(y[0, 200:, 5]).all())
    assert bool(torch.isfinite(y[0, :300, 7]).all()) and bool(torch.isnan(y[0, 300:, 7]).all())
    assert float(y[0, 100, 8]) == float(y[0, 99, 8]) and bool(torch.isfinite(y[..., [8, 9]]).all())
    g = sc.gated_scan_grad(torch.ones_like(y), x2, f2, starts, rate2, i)
    assert float(g["drate"][1]) == 0 and float(g["drate"][2]) == 0
    for name in ("dx", "dforget", "dinput_gate"):
        assert bool(torch.isfinite(g[name][..., [0, 1, 2, 3, 4, 6, 8, 9, 10, 11]]).all()), name
    assert bool(torch.isfinite(g["drate"][[0, 1, 2, 3, 4, 6, 8, 9, 10, 11]]).all())
    del clean


def test_states_beyond_a_chunks_decay():
    # a state of 1e30 and decays whose product over a run leaves float32's range
    b, l, d = 1, 600, 6
    x = torch.zeros(b, l, d, device="cuda")
    f = torch.full((b, l, d), -0.5, device="cuda")
    init = torch.full((b, d), 1e30, device="cuda")
    y, state = sc.gated_scan(x, f, initial_state=init)
    a = 1 / (1 + math.exp(0.5))
    want = 1e30 * torch.tensor(a, dtype=torch.float64) ** torch.arange(1, l + 1, dtype=torch.float64)
    got = y[0, :, 0].double().cpu()
    ok = want > 1e-30
    assert int(ok.sum()) > 130
    # one rounding a token, and 1.5e-7 of the gate's own
    assert bool(((got - want).abs()[ok] <= want[ok] * 4e-7 * torch.arange(1, l + 1)[ok]).all())
    assert bool((got[~ok] <= 1e-29).all()) and bool((got >= 0).all())
    inf = torch.full((b, d), float("inf"), device="cuda")
    y, state = sc.gated_scan(x, f, initial_state=inf)
    assert bool(torch.isinf(y).all()) and bool(torch.isinf(state).all())


@pytest.mark.parametrize("l", [3, 131])
def test_more_sequences_than_an_axis_holds(l):
    # 65535 sequences a launch: the ones at its end and behind it, in one tile and in several
    b, d = 65538, 3
    r = torch.Generator(device="cuda").manual_seed(l)
    x, f = (torch.randn((b, l, d), generator=r, device="cuda") for _ in range(2))
    rate = torch.rand(d, generator=r, device="cuda")
    init = torch.randn((b, d), generator=r, device="cuda")
    y, state, starts = sc.gated_scan(x, f, rate, initial_state=init, keep_starts=True)
    g = sc.gated_scan_grad(x, x, f, starts, rate)
    total = torch.zeros(d, dtype=torch.float64, device="cuda")
    for lo, hi in ((0, 40000), (40000, b)):
        s = slice(lo, hi)
        y2, state2, starts2 = sc.gated_scan(x[s], f[s], rate, initial_state=init[s].contiguous(), keep_starts=True)
        g2 = sc.gated_scan_grad(x[s], x[s], f[s], starts2, rate)
        assert torch.equal(y[s], y2) and torch.equal(state[s], state2)
        assert all(torch.equal(g[n][s], g2[n]) for n in ("dx", "dforget", "dstate"))
        total += g2["drate"].double()
    # (sums of 2^16 x l terms in another order: 16 strands of 4096 tiles, some 2^12 roundings of a sum)
    size = (g["dforget"].double().abs().sum((0, 1)) / rate).clamp(min=1.0)
    assert bool(((g["drate"].double() - total).abs() <= size * 2.0 ** -12 * 8).all())


def test_more_runs_than_an_axis_holds():
    # one channel, tiles beyond 65535 in both directions: the whole against its parts
    l, cut = 8_500_000, 5_000_001
    r = torch.Generator(device="cuda").manual_seed(5)
    x, f = (torch.randn((1, l, 1), generator=r, device="cuda").bfloat16() for _ in range(2))
    rate = torch.full((1,), 1e-3, device="cuda")
    y, state, starts = sc.gated_scan(x, f, rate, keep_starts=True)
    g = sc.gated_scan_grad(x, x, f, starts, rate)
    y1, mid, starts1 = sc.gated_scan(x[:, :cut], f[:, :cut], rate, keep_starts=True)
    y2, last, starts2 = sc.gated_scan(x[:, cut:], f[:, cut:], rate, initial_state=mid, keep_starts=True)
    g2 = sc.gated_scan_grad(x[:, cut:], x[:, cut:], f[:, cut:], starts2, rate)
    g1 = sc.gated_scan_grad(x[:, :cut], x[:, :cut], f[:, :cut], starts1, rate, dfinal=g2["dstate"])
    # states of about 30 (1 over the root of the rate) that differ by roundings of 2^-24 over some thousand tokens
    near = lambda a, b: bool(((a.float() - b.float()).abs() <= a.float().abs() * 2.0 ** -7 + 1e-2).all())  # noqa: E731
    assert near(y, torch.cat([y1, y2], 1)) and near(state, last)
    assert near(g["dx"], torch.cat([g1["dx"], g2["dx"]], 1)) and near(g["dstate"], g1["dstate"])
    # where a part begins with the whole, it is the same to the bit
    assert torch.equal(y[:, :4096], y1[:, :4096])


def test_a_state_that_never_comes():
    # a build that asks for a state once and then takes it as lost: the call ends, the first tile is right and
    # what follows is right or no number
    from stream_compaction_amd import build
    from stream_compaction_amd.sequence import _gated_args
    k, _ = inputs((2, 900, 300, "f32", None, "rate in"), 160)
    want, _ = sc.gated_scan(**k)
    L = sc.load(build.FALLBACK_LIB_PATH)
    a = _gated_args(k["x"], k["forget"], k["rate"], k["input_gate"], None, None, None, False)
    y = torch.empty_like(want)
    scratch = torch.empty(L.gated_scan_scratch_bytes(a), dtype=torch.uint8, device="cuda")
    sc.check(L.gated_scan(a, y.data_ptr(), None, None, scratch.data_ptr(), scratch.numel(),
                          torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(y[:, :128], want[:, :128])
    lost = torch.isnan(y)
    assert torch.equal(y[~lost], want[~lost])


def test_refusals_leave_outputs():
    x = torch.randn(2, 8, 16, device="cuda")
    rate = torch.rand(16, device="cuda")
    for call in (lambda: sc.gated_scan(x, x, out=x), lambda: sc.gated_scan(x, x, rate=rate.half()),
                 lambda: sc.gated_scan(x, x[:, :7]), lambda: sc.gated_scan(x, x.transpose(1, 2)),
                 lambda: sc.gated_scan(x, x, lengths=torch.tensor([1, 2], device="cuda")),
                 lambda: sc.gated_scan(x, x.cpu()), lambda: sc.gated_scan(x.cpu(), x),
                 lambda: sc.gated_scan_grad(x, x, x, torch.zeros(5, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(NotImplementedError):
        sc.gated_scan(x.double(), x.double())
    assert bool(torch.isfinite(x).all()) and host(x).shape == (2, 8, 16)
