"""Causal convolution, selective scan and token embedding on the GPU against the
float64 oracle of ``sequence_ref`` (whose bounds count float32 roundings), over
the sizes, masks, strides and types where the kernels can go wrong; and each
gradient and step against the operator it belongs to."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
import stream_compaction_amd as sc

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def act(g, shape, dt, scale=1.0):
    """An activation on the GPU and its exact float64 values."""
    t = (torch.randn(shape, generator=g) * scale).to(TYPES[dt])
    return t.cuda(), t.double().numpy()


def par(g, shape, scale=1.0, shift=0.0):
    t = torch.randn(shape, generator=g) * scale + shift
    return t.cuda(), t.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def agree(got, want, dt, what):
    worst = ref.excess(host(got), want, dt)
    assert worst == 0.0, f"{what}: {worst:.3g} times the bound"


def poison(t, lengths):
    """NaN and infinities where no token exists."""
    if lengths is not None:
        for i, n in enumerate(lengths):
            n = min(max(n, 0), t.shape[1])
            t[i, n:] = float("nan")
            t[i, n::2] = float("inf")
    return t


# batch, length, channels, states, groups, type, lengths (None: all), options
SCANS = [
    (1, 1, 1, 1, 1, "f32", None, ""),
    (1, 1, 16, 16, 1, "bf16", None, "gate soft bias D init"),
    (2, 0, 5, 4, 1, "f32", None, "init"),
    (1, 63, 16, 16, 1, "bf16", None, "gate soft bias D"),
    (2, 64, 17, 13, 1, "f32", None, "gate soft bias D init"),
    (1, 65, 33, 16, 3, "f16", None, "soft bias"),
    (2, 128, 24, 8, 2, "bf16", [128, 37], "gate D init"),
    (1, 129, 16, 16, 1, "f32", None, "soft D"),
    (3, 200, 40, 5, 1, "bf16", [0, 200, 1], "gate soft bias D init"),
    (1, 256, 18, 17, 1, "f16", None, "gate soft bias D init"),
    (1, 257, 20, 3, 1, "f32", None, "gate"),
    (2, 512, 16, 16, 1, "bf16", [512, 511], "soft bias D"),
    (2, 513, 18, 16, 2, "f16", [513, 512], "gate soft bias D init"),
    (1, 1100, 34, 16, 1, "bf16", None, "gate soft bias D init"),
    (1, 30, 8, 64, 1, "f32", None, "gate soft bias D init"),
    (1, 300, 6, 33, 1, "bf16", None, "gate soft bias D init"),
    (5, 70, 19, 16, 19, "f32", [70, -3, 0, 900, 64], "soft init"),
]


def scan_inputs(case, seed, grads=False):
    b, l, d, n, g, dt, lengths, opts = case
    r = gen(seed)
    k, w = {}, {}
    k["x"], w["x"] = act(r, (b, l, d), dt)
    soft = "soft" in opts
    k["dt"], w["dt"] = act(r, (b, l, d), dt, 0.5)
    if not soft:        # steps as a layer gives them: small and positive
        k["dt"] = (k["dt"].abs() * 0.1)
        w["dt"] = host(k["dt"])
    A = -torch.rand((d, n), generator=r) * 4 - 0.01
    k["A"], w["A"] = A.cuda(), A.double().numpy()
    k["B"], w["B"] = act(r, (b, l, g, n), dt)
    k["C"], w["C"] = act(r, (b, l, g, n), dt)
    w.update(D=None, z=None, dt_bias=None, initial=None)
    if "D" in opts:
        k["D"], w["D"] = par(r, (d,))
    if "gate" in opts:
        k["z"], w["z"] = act(r, (b, l, d), dt)
    if "bias" in opts:
        k["dt_bias"], w["dt_bias"] = par(r, (d,), 0.5, -3.0)
    if "init" in opts:
        k["initial_state"], w["initial"] = par(r, (b, d, n))
    if lengths is not None:
        for name in ("x", "dt", "B", "C", "z"):
            if name in k:
                poison(k[name], lengths)
        k["lengths"] = torch.tensor(lengths, dtype=torch.int32).cuda()
        w["lengths"] = np.minimum(np.array(lengths), l)
    k["softplus"] = soft
    w["soft"] = soft
    if grads:
        dy, w["dy"] = act(r, (b, l, d), dt)
        dfinal, w["dfinal"] = par(r, (b, d, n))
        return k, w, poison(dy, lengths), dfinal
    return k, w


@pytest.mark.parametrize("case", SCANS, ids=[f"{c[:6]}".replace(" ", "") for c in SCANS])
def test_scan(case):
    k, w = scan_inputs(case, 10)
    y, state = sc.selective_scan(**k)
    want = ref.scan(**w)
    agree(y, want["y"], case[5], "y")
    agree(state, want["state"], "f32", "state")


@pytest.mark.parametrize("case", SCANS, ids=[f"{c[:6]}".replace(" ", "") for c in SCANS])
def test_scan_grad(case):
    k, w, dy, dfinal = scan_inputs(case, 20, grads=True)
    y, state, starts = sc.selective_scan(keep_starts=True, **k)
    k.pop("initial_state", None)
    got = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    again = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    want = ref.scan(**w)
    agree(y, want["y"], case[5], "y")
    for name in ("dx", "ddt", "dz", "dB", "dC"):
        if got[name] is not None:
            agree(got[name], want[name], case[5], name)
    for name in ("dA", "dD", "ddt_bias", "dstate"):
        if got[name] is not None:
            agree(got[name], want[name], "f32", name)
    assert (got["dz"] is None) == ("z" not in k) and (got["dD"] is None) == ("D" not in k)
    for name, v in got.items():
        assert v is None or torch.equal(v, again[name]), f"{name} differs from call to call"


def strided(t, how):
    """The same values laid out as a view of something larger."""
    if how == "halves":                    # one half of a wider row
        big = torch.full(t.shape[:-1] + (2 * t.shape[-1],), float("nan"), dtype=t.dtype, device="cuda")
        big[..., t.shape[-1]:] = t
        return big[..., t.shape[-1]:]
    if how == "shifted":                   # one element off every alignment
        big = torch.full((t.numel() + 1,), float("nan"), dtype=t.dtype, device="cuda")
        v = big[1:].view(t.shape)
        v.copy_(t)
        return v
    if how == "time_major":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    raise KeyError(how)


@pytest.mark.parametrize("how", ["halves", "shifted", "time_major"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides(how, dt):
    case = (2, 130, 48, 16, 2, dt, [130, 77], "gate soft bias D init")
    k, _, dy, dfinal = scan_inputs(case, 30, grads=True)
    y, state, starts = sc.selective_scan(keep_starts=True, **k)
    s = {n: strided(v, how) if n in ("x", "dt", "B", "C", "z") else v for n, v in k.items()}
    y2, state2, starts2 = sc.selective_scan(keep_starts=True, **s)
    assert torch.equal(y, y2) and torch.equal(state, state2)
    init = k.pop("initial_state")
    s.pop("initial_state")
    g1 = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    g2 = sc.selective_scan_grad(strided(dy, how), starts=starts2, dfinal=dfinal, **s)
    for name in g1:
        assert torch.equal(g1[name], g2[name]), name
    # the convolution's and the embedding's rows
    r = gen(31)
    w, bias = par(r, (48, 4))[0], par(r, (48,))[0]
    cs, ln = act(r, (2, 3, 48), dt)[0], k["lengths"]
    a = sc.causal_conv(k["x"], w, bias, cs, ln)
    b = sc.causal_conv(s["x"], w, bias, cs, ln)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = sc.causal_conv_grad(dy, k["x"], w, bias, cs, ln)
    gb = sc.causal_conv_grad(strided(dy, how), s["x"], w, bias, cs, ln)
    assert torch.equal(ga["dx"], gb["dx"]) and torch.equal(ga["dstate"], gb["dstate"])
    # (filter sums may group lanes otherwise where rows are not aligned)
    wide = {"dweight": None, "dbias": None}
    for name in wide:
        assert torch.allclose(ga[name], gb[name], rtol=0, atol=260 * 2.0 ** -22 * 8)
    if how != "time_major":
        table = act(r, (97, 48), dt)[0]
        ids = torch.randint(-2, 99, (2, 130), generator=r).cuda()
        e1 = sc.embedding(table, ids, scale=3.0)
        assert torch.equal(e1, sc.embedding(strided(table, how), ids, scale=3.0))
    del init


def test_broadcast_strides():
    # one token of dt and one batch of B and C, repeated with stride 0
    case = (3, 70, 20, 8, 1, "f32", None, "gate D")
    k, _ = scan_inputs(case, 40)
    k["dt"] = k["dt"][:, :1].expand(3, 70, 20)
    k["B"], k["C"] = k["B"][:1].expand(3, -1, -1, -1), k["C"][:1].expand(3, -1, -1, -1)
    y, state = sc.selective_scan(**k)
    full = {n: v.contiguous() if torch.is_tensor(v) else v for n, v in k.items()}
    y2, state2 = sc.selective_scan(**full)
    assert torch.equal(y, y2) and torch.equal(state, state2)


def test_scan_in_parts_and_steps():
    # a sequence scanned in two parts, then token by token, is the whole one's
    case = (2, 150, 37, 16, 1, "f32", None, "gate soft bias D init")
    k, w = scan_inputs(case, 50)
    want = ref.scan(**w)
    cut = 90
    part = {n: k[n][:, :cut] for n in ("x", "dt", "B", "C", "z")}
    y1, mid = sc.selective_scan(**{**k, **part})
    agree(y1, ref.V(want["y"].val[:, :cut], want["y"].mag[:, :cut], want["y"].err[:, :cut]), "f32", "first part")
    ys = []
    step = {n: k[n] for n in ("A", "D", "dt_bias", "softplus")}
    for t in range(cut, 150):
        tok = {n: k[n][:, t] for n in ("x", "dt", "B", "C", "z")}
        ys.append(sc.selective_scan_step(mid, **tok, **step))
    rest = torch.stack(ys, 1)
    agree(rest, ref.V(want["y"].val[:, cut:], want["y"].mag[:, cut:], want["y"].err[:, cut:]), "f32", "steps")
    agree(mid, want["state"], "f32", "state")


STEPS = [(1, 1, 1, 1, "f32"), (3, 17, 13, 1, "bf16"), (2, 40, 16, 2, "f16"), (130, 64, 16, 1, "bf16"),
         (2, 24, 64, 3, "f32"), (4, 33, 33, 1, "f32"), (1, 4096, 16, 1, "bf16"), (2, 48, 8, 4, "f16"), (3, 7, 4, 1, "bf16")]


@pytest.mark.parametrize("b,d,n,g,dt", STEPS)
@pytest.mark.parametrize("opts", ["", "gate soft bias D"])
def test_scan_step(b, d, n, g, dt, opts):
    case = (b, 1, d, n, g, dt, None, opts + " init")
    k, w = scan_inputs(case, 60)
    want = ref.scan(**w)
    state = k.pop("initial_state")
    tok = {name: (v[:, 0] if name in ("x", "dt", "B", "C", "z") else v) for name, v in k.items()}
    before, fresh = state.clone(), torch.empty_like(state)
    y = sc.selective_scan_step(state, new_state=fresh, **tok)
    assert torch.equal(state, before)
    agree(y, ref.V(want["y"].val[:, 0], want["y"].mag[:, 0], want["y"].err[:, 0]), dt, "y")
    agree(fresh, want["state"], "f32", "state")
    y2 = sc.selective_scan_step(state, **tok)
    assert torch.equal(y, y2) and torch.equal(state, fresh)


# batch, length, channels, width, type, lengths, silu, bias and state
CONVS = [
    (1, 1, 1, 1, "f32", None, True, True), (1, 1, 8, 4, "bf16", None, True, True),
    (2, 0, 9, 4, "f32", None, True, True), (2, 2, 16, 4, "bf16", [2, 1], True, True),
    (3, 15, 24, 4, "f16", [15, 0, 2], True, True), (1, 16, 7, 3, "f32", None, False, True),
    (2, 17, 520, 4, "bf16", None, True, False), (1, 35, 64, 8, "bf16", [33], True, True),
    (2, 64, 12, 2, "f32", [64, 63], False, False), (2, 131, 40, 5, "f16", None, True, True),
    (5, 33, 257, 6, "f32", [33, -1, 0, 50, 4], True, True), (1, 300, 16, 7, "bf16", None, True, True),
    (2, 1, 8, 1, "f16", None, False, True),
]


def conv_inputs(case, seed):
    b, l, d, w, dt, lengths, act_on, more = case
    r = gen(seed)
    x, xr = act(r, (b, l, d), dt)
    weight, wr = par(r, (d, w), 0.5)
    bias, br = par(r, (d,)) if more else (None, None)
    init, ir = act(r, (b, w - 1, d), dt) if more else (None, None)
    ln = None
    if lengths is not None:
        poison(x, lengths)
        ln = torch.tensor(lengths, dtype=torch.int32).cuda()
    dy, dyr = act(r, (b, l, d), dt)
    df, dfr = act(r, (b, w - 1, d), dt)
    poison(dy, lengths)
    return (x, weight, bias, init, ln, act_on), (xr, wr, br, ir, lengths, act_on), (dy, dyr), (df, dfr)


@pytest.mark.parametrize("case", CONVS, ids=[f"{c[:5]}".replace(" ", "") for c in CONVS])
def test_conv(case):
    dt = case[4]
    dev, cpu, (dy, dyr), (df, dfr) = conv_inputs(case, 70)
    x, weight, bias, init, ln, act_on = dev
    # a lane adds 16 tokens a run, 4 waves, then the sets in four strands
    want = ref.conv(*cpu, dy=dyr, dfinal=dfr, depth=16 * (1 + case[0] * case[1] // 4096) + 8 + 4 + case[0] * case[1] // 256)
    y, state = sc.causal_conv(x, weight, bias, init, ln, act_on)
    agree(y, want["y"], dt, "y")
    assert np.array_equal(host(state), want["state"].val)
    got = sc.causal_conv_grad(dy, x, weight, bias, init, ln, act_on, dfinal=df)
    again = sc.causal_conv_grad(dy, x, weight, bias, init, ln, act_on, dfinal=df)
    agree(got["dx"], want["dx"], dt, "dx")
    agree(got["dweight"], want["dweight"], "f32", "dweight")
    if bias is not None:
        agree(got["dbias"], want["dbias"], "f32", "dbias")
        agree(got["dstate"], want["dstate"], dt, "dstate")
    for name, v in got.items():
        assert v is None or torch.equal(v, again[name]), f"{name} differs from call to call"


@pytest.mark.parametrize("case", [c for c in CONVS if c[1] > 0], ids=[f"{c[:5]}".replace(" ", "") for c in CONVS if c[1] > 0])
def test_conv_step(case):
    b, l, d, w, dt, _, act_on, more = case
    (x, weight, bias, init, _, _), _, _, _ = conv_inputs((b, l, d, w, dt, None, act_on, more), 80)
    want, last = sc.causal_conv(x, weight, bias, init, silu=act_on)
    state = torch.zeros(b, w - 1, d, dtype=x.dtype, device="cuda") if init is None else init.clone()
    for t in range(min(l, 20)):
        before, fresh = state.clone(), torch.empty_like(state)
        y = sc.causal_conv_step(state, x[:, t], weight, bias, silu=act_on, new_state=fresh)
        assert torch.equal(state, before)
        y2 = sc.causal_conv_step(state, x[:, t], weight, bias, silu=act_on)
        assert torch.equal(y, y2) and torch.equal(fresh, state)
        # the same products in the same order
        assert torch.equal(y, want[:, t])
    if l <= 20:
        assert torch.equal(state, last)


# tokens shape, rows, channels, type, gradient type, ids: "mixed", "one" row, "masked" all
EMBEDS = [
    ((0,), 7, 8, "f32", "f32", "mixed"), ((1,), 1, 1, "f32", "f32", "mixed"),
    ((2, 3), 5, 16, "bf16", "bf16", "mixed"), ((33,), 300, 9, "f16", "f16", "mixed"),
    ((64,), 70000, 24, "bf16", "f32", "mixed"), ((1000,), 3, 520, "bf16", "bf16", "mixed"),
    ((4, 513), 257, 33, "f32", "f32", "mixed"), ((3000,), 100, 136, "f16", "f32", "one"),
    ((130,), 255, 40, "bf16", "bf16", "masked"), ((5000,), 256, 64, "f32", "f32", "mixed"),
    ((20000,), 40, 8, "bf16", "f32", "one"),
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("case", EMBEDS, ids=[f"{c[:5]}".replace(" ", "") for c in EMBEDS])
def test_embedding(case, wide):
    shape, rows, d, dt, odt, kind = case
    r = gen(90)
    table, tr = act(r, (rows, d), dt)
    ids = torch.randint(-1, rows + 1, shape, generator=r)
    if kind == "one":
        ids = torch.where(torch.rand(shape, generator=r) < 0.9, torch.full_like(ids, rows // 2), ids)
    if kind == "masked":
        ids = torch.where(ids % 2 == 0, torch.full_like(ids, -2 ** 31), torch.full_like(ids, 2 ** 31 - 1))
    ids = ids if wide else ids.int()
    dout, dr = act(r, shape + (d,), dt)
    idn = ids.numpy().astype(np.int64)
    bad = torch.tensor((idn < 0) | (idn >= rows))
    dout[bad.cuda()] = float("nan")
    got = sc.embedding(table, ids.cuda(), scale=1.75)
    agree(got, ref.embedding(tr, idn, 1.75), dt, "rows")
    flat = idn.reshape(-1)
    # 32 tokens a segment, then the segments of a run
    longest = np.bincount(flat[(flat >= 0) & (flat < rows)], minlength=1).max() if flat.size else 0
    want = ref.embedding_grad(dr.reshape(-1, d), flat, rows, 1.75, 34 + longest // 32)
    g = sc.embedding_grad(dout, ids.cuda(), rows, scale=1.75, dtype=TYPES[odt])
    assert g.dtype == TYPES[odt]
    agree(g, want, odt, "table gradient")
    assert torch.equal(g, sc.embedding_grad(dout, ids.cuda(), rows, scale=1.75, dtype=TYPES[odt]))


def test_embedding_grad_unaligned_output():
    r = gen(95)
    dout, dr = act(r, (50, 21), "bf16")
    ids = torch.randint(0, 30, (50,), generator=r)
    big = torch.full((30 * 21 + 40,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[3:3 + 30 * 21].view(30, 21)
    sc.embedding_grad(dout, ids.cuda(), 30, out=out)
    agree(out, ref.embedding_grad(dr, ids.numpy(), 30, 1.0, 51), "bf16", "gradient")
    assert bool((big[:3] == 7).all()) and bool((big[3 + 30 * 21:] == 7).all())


def test_far_offsets():
    # strides that pass 2^31 elements and 2^32 bytes
    step = (1 << 30) + 8
    big = torch.zeros(2 * step + 64, dtype=torch.bfloat16, device="cuda")
    r = gen(100)
    x0 = act(r, (1, 3, 16), "bf16")[0]
    far = big.as_strided((1, 3, 16), (3 * step, step, 1))
    far.copy_(x0)
    w, bias = par(r, (16, 3))[0], par(r, (16,))[0]
    assert torch.equal(sc.causal_conv(far, w, bias)[0], sc.causal_conv(x0, w, bias)[0])
    a, b = sc.causal_conv_grad(far, far, w, bias), sc.causal_conv_grad(x0, x0, w, bias)
    assert all(torch.equal(a[n], b[n]) for n in ("dx", "dweight", "dbias"))
    A = -torch.rand((16, 16), generator=r).cuda()
    Bf = big.as_strided((1, 3, 1, 16), (3 * step, step, 16, 1))
    B0 = x0[:, :, None].contiguous()
    y1, s1, k1 = sc.selective_scan(far, far, A, Bf, Bf, z=far, softplus=True, keep_starts=True)
    y0, s0, k0 = sc.selective_scan(x0, x0, A, B0, B0, z=x0, softplus=True, keep_starts=True)
    assert torch.equal(y1, y0) and torch.equal(s1, s0)
    g1 = sc.selective_scan_grad(far, far, far, A, Bf, Bf, k1, z=far, softplus=True)
    g0 = sc.selective_scan_grad(x0, x0, x0, A, B0, B0, k0, z=x0, softplus=True)
    for n in ("dx", "ddt", "dz", "dB", "dC", "dA"):
        assert torch.equal(g1[n], g0[n]), n
    table = big.as_strided((3, 16), (step, 1))
    ids = torch.tensor([2, 0, 1, 2, 5], device="cuda")
    assert torch.equal(sc.embedding(table, ids, scale=2.0), sc.embedding(x0[0], ids, scale=2.0))
    del big, far, Bf, table
    torch.cuda.empty_cache()


def test_another_stream():
    case = (2, 300, 48, 16, 1, "bf16", [300, 111], "gate soft bias D init")
    k, _, dy, dfinal = scan_inputs(case, 110, grads=True)
    y, state, starts = sc.selective_scan(keep_starts=True, **k)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, state2, starts2 = sc.selective_scan(keep_starts=True, **k)
        k.pop("initial_state")
        g2 = sc.selective_scan_grad(dy, starts=starts2, dfinal=dfinal, **k)
    s.synchronize()
    g = sc.selective_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(state, state2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


def test_graph_replays():
    # one graph of the whole path, replayed on new inputs with eager work between
    d, n, rows = 48, 16, 301
    r = gen(120)
    table = act(r, (rows, d), "bf16")[0]
    w, bias = par(r, (d, 4))[0], par(r, (d,))[0]
    A = -torch.rand((d, n), generator=r).cuda()
    D = par(r, (d,))[0]
    ids = torch.randint(-1, rows, (2, 140), generator=r).cuda()
    dt, B, C = (act(r, s, "bf16", 0.3)[0] for s in ((2, 140, d), (2, 140, 1, n), (2, 140, 1, n)))
    dy = act(r, (2, 140, d), "bf16")[0]

    def work():
        e = sc.embedding(table, ids, scale=2.0)
        u, cs = sc.causal_conv(e, w, bias)
        y, state, starts = sc.selective_scan(u, dt, A, B, C, D, softplus=True, keep_starts=True)
        g = sc.selective_scan_grad(dy, u, dt, A, B, C, starts, D, softplus=True)
        gc = sc.causal_conv_grad(g["dx"], e, w, bias)
        gt = sc.embedding_grad(gc["dx"], ids, rows, scale=2.0, dtype=torch.float32)
        cs2, st2 = cs.clone(), state.clone()
        v = sc.causal_conv_step(cs2, e[:, 0], w, bias)
        z = sc.selective_scan_step(st2, v, dt[:, 0], A, B[:, 0], C[:, 0], D, softplus=True)
        return [y, state, g["dA"], g["dB"], g["ddt"], gc["dweight"], gc["dbias"], gt, z, st2, cs2]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        ids.copy_(torch.randint(-1, rows, (2, 140), generator=r))
        dy.copy_(torch.randn((2, 140, d), generator=r))
        want = [t.clone() for t in work()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"replay {i}, output {j}"


def test_refusals_leave_outputs():
    x = torch.randn(2, 8, 16, device="cuda")
    w = torch.randn(16, 4, device="cuda")
    with pytest.raises(ValueError):
        sc.causal_conv(x, w, out=x)                                  # in place
    with pytest.raises(NotImplementedError):
        sc.causal_conv(x, torch.randn(16, 9, device="cuda"))         # width
    with pytest.raises(NotImplementedError):
        sc.causal_conv(x.double(), w)
    with pytest.raises(ValueError):
        sc.causal_conv(x.transpose(1, 2), torch.randn(8, 4, device="cuda"))   # channels not contiguous
    with pytest.raises(ValueError):
        sc.causal_conv(x, w.half())
    with pytest.raises(ValueError):
        sc.causal_conv(x, w, lengths=torch.tensor([1, 2], device="cuda"))      # int64 lengths
    A = -torch.rand(16, 65, device="cuda")
    BC = torch.randn(2, 8, 1, 65, device="cuda")
    with pytest.raises(NotImplementedError):
        sc.selective_scan(x, x, A, BC, BC)                           # states
    A, BC = -torch.rand(16, 4, device="cuda"), torch.randn(2, 8, 3, 4, device="cuda")
    with pytest.raises(ValueError):
        sc.selective_scan(x, x, A, BC, BC)                           # groups do not divide
    with pytest.raises(ValueError):
        sc.selective_scan(x, x, A, BC[:, :, :1], BC[:, :, :2])
    with pytest.raises(ValueError):
        sc.selective_scan(x.cpu(), x, A, BC, BC)
    with pytest.raises(ValueError):
        sc.selective_scan_grad(x, x, x, A, BC[:, :, :1], BC[:, :, :1], torch.zeros(3, device="cuda"))
    with pytest.raises(NotImplementedError):
        sc.embedding(x[0], torch.tensor([1.0], device="cuda"))
    with pytest.raises(ValueError):
        sc.embedding(x[0], torch.tensor([1]))                        # ids on the host
    with pytest.raises(NotImplementedError):
        sc.embedding_grad(x[0], torch.arange(8, device="cuda"), 9, dtype=torch.float16)
    with pytest.raises(ValueError):
        sc.embedding_grad(x[0], torch.arange(8, device="cuda"), 9, scratch=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert bool(torch.isfinite(x).all())
