"""Beam search on the GPU against the float64 oracle of ``beam_ref``: choices are equal, scores are
within a float32 rounding of it; states move to the bit."""
import math

import numpy as np
import pytest
import torch

import beam_ref as ref
import stream_compaction_amd as sc
from test_gpu_sequence import TYPES, gen, strided

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(logits, scores, count, finished=None, end=0, what="", **more):
    """The call against the oracle; scores to half a step of float32, and 1e-9 for a sum and
    exponentials in 64 bits that are good to 4e-11 each."""
    f = None if finished is None else finished.cuda()
    got = sc.beam_select(logits, scores.cuda(), count, finished=f, end_token=end, **more)
    want = ref.select(logits.double().cpu().numpy(), scores.double().numpy(), count,
                      None if finished is None else finished.numpy(), end)
    assert np.array_equal(got[1].cpu().numpy(), want[1]), f"{what} parents"
    assert np.array_equal(got[2].cpu().numpy(), want[2]), f"{what} tokens"
    a, b = got[0].double().cpu().numpy(), want[0]
    low = np.isinf(b)
    assert np.array_equal(a[low], b[low]), f"{what} infinite scores"
    assert (np.abs(a[~low] - b[~low]) <= np.abs(b[~low]) * 2.0 ** -24 + 1e-9).all(), f"{what} scores"
    again = sc.beam_select(logits, scores.cuda(), count, finished=f, end_token=end, **more)
    assert all(torch.equal(x, y) for x, y in zip(got, again)), f"{what} differs from call to call"
    return got


def normal(g, shape, dt, scale=2.0):
    return (torch.randn(shape, generator=g) * scale).to(TYPES[dt]).cuda()


# batch, beams, vocabulary, count, type
CASES = [(1, 1, 1, 1, "f32"), (1, 1, 3, 3, "bf16"), (2, 3, 2, 6, "f16"), (3, 2, 7, 5, "bf16"), (1, 4, 8, 8, "bf16"),
         (2, 5, 9, 11, "f32"), (1, 1, 255, 64, "f32"), (2, 2, 2047, 4, "bf16"), (1, 3, 2048, 6, "f16"),
         (1, 2, 2049, 64, "bf16"), (1, 4, 32003, 4, "bf16"), (5, 8, 8193, 16, "f16"), (2, 16, 5000, 33, "f32"),
         (1, 64, 1111, 64, "bf16"), (3, 13, 4097, 27, "f32"), (40, 8, 20001, 16, "bf16"), (70, 8, 9001, 8, "f32"),
         (130, 4, 30000, 8, "f16"), (1, 1, 130000, 2, "f32"), (300, 1, 40, 40, "bf16")]


@pytest.mark.parametrize("ended", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[str(c).replace(" ", "") for c in CASES])
def test_select(case, ended):
    b, k, v, n, dt = case
    g = gen(b * 1000 + v)
    logits = normal(g, (b, k, v), dt)
    scores = -torch.rand((b, k), generator=g) * 3
    finished = (torch.rand((b, k), generator=g) < 0.4).to(torch.uint8) if ended else None
    check(logits, scores, n, finished, v // 2)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", ["equal", "two values", "lowest", "few", "runs", "falling", "rising", "masked row", "zeros"])
def test_ties_and_masks(how, dt):
    # where what is above a bound, or equal to it, is much; most of it in one lane, segment or beam
    b, k, v, n = 2, 4, 20011, 9
    g = gen(7)
    x = torch.randn((b, k, v), generator=g)
    lowest = torch.finfo(TYPES[dt]).min
    if how == "equal":
        x[:] = 1.25
    elif how == "two values":
        x = (torch.rand((b, k, v), generator=g) < 0.3).float() * 2 - 1
    elif how == "lowest":                                # all but a few at the type's lowest value
        keep = torch.rand((b, k, v), generator=g) < 2e-4
        x = torch.where(keep, x, torch.full_like(x, lowest))
    elif how == "few":                                   # fewer than asked for have a chance
        x[:] = -INF
        x[0, 2, 17], x[0, 0, 19000], x[0, 0, 3], x[1, 3, v - 1] = 1.0, 2.0, -1.0, 0.5
    elif how == "runs":                                  # the greatest side by side, in steps the type tells apart
        x = x.clamp(max=2)
        x[:, :, 5000:7500] = 8 + torch.arange(2500) / 512
        x[:, 1] -= 1
    elif how == "falling":
        x = (-torch.arange(v).float() / 1000).expand(b, k, v).clone()
    elif how == "rising":
        x = (torch.arange(v).float() / 1000).expand(b, k, v).clone()
    elif how == "masked row":
        x[0, 0], x[0, 3], x[1] = -INF, float("nan"), -INF
        x[1, 2, 11] = 0.0
    else:
        x = torch.where(torch.rand((b, k, v), generator=g) < 0.5, torch.tensor(0.0), torch.tensor(-0.0))
    scores = torch.tensor([[0.0, -0.5, 0.0, -1.0]]).repeat(b, 1)
    check(x.to(TYPES[dt]).cuda(), scores, n, what=how)
    check(x.to(TYPES[dt]).cuda(), scores, 64, what=how)
    check(x.to(TYPES[dt]).cuda(), torch.zeros(b, k), 2, what=how)


def test_equal_beams_lie_anywhere():
    # beams alike in all but where their rows begin (odd vocabulary, one element off alignment): the lower goes first
    g = gen(8)
    for dt, v in (("bf16", 40003), ("f16", 9), ("f32", 5001), ("bf16", 6)):
        row = normal(g, (1, 1, v), dt)
        x = strided(row.expand(2, 8, v).contiguous(), "shifted")
        got = check(x, torch.zeros(2, 8), 16, what=dt)
        assert got[1][:, :8].tolist() == [list(range(8))] * 2
        assert bool((got[0][:, :8] == got[0][:, :1]).all())


def test_infinite_logits_and_scores():
    g = gen(9)
    x = torch.randn((1, 6, 3000), generator=g)
    x[0, 0, 2999] = INF
    x[0, 1, 5], x[0, 1, 2500] = INF, INF
    x[0, 2, 7] = float("nan")
    scores = torch.tensor([[-1.0, -1.5, 0.0, -INF, float("nan"), 0.25]])
    for n in (4, 12, 64):
        check(x.cuda(), scores, n)
    scores[0, 3] = INF
    check(x.cuda(), scores, 20)
    done = torch.tensor([[1, 0, 0, 1, 1, 0]], dtype=torch.uint8)
    check(x.cuda(), torch.tensor([[-INF, 0.0, 0.0, 0.5, float("nan"), 0.0]]), 20, done, 2999)
    check(torch.full((1, 2, 30), -INF).cuda(), torch.zeros(1, 2), 40, torch.tensor([[0, 1]], dtype=torch.uint8), 4)


def test_close_scores():
    # beams whose scores differ by less than float32 tells apart in a sum over the vocabulary
    g = gen(10)
    v = 30000
    row = torch.randn((1, 1, v), generator=g).expand(1, 4, v).contiguous()
    row[0, 1:, 100] -= 1.0                               # sums that differ in their 7th digit
    row[0, 2:, 200] -= 1e-3
    row[0, 3, 300] += 1e-4
    for dt in ("f32",):
        check(row.to(TYPES[dt]).cuda(), torch.zeros(1, 4), 32, what=dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_streams(dt):
    g = gen(11)
    b, k, v, n = 3, 4, 3001, 8
    x = normal(g, (b, k, v), dt)
    scores = -torch.rand((b, k), generator=g)
    want = check(x, scores, n)
    wide = torch.full((b, k, 2 * v + 3), 99.0, dtype=x.dtype, device="cuda")
    wide[..., 3:v + 3] = x
    for y in (wide[..., 3:v + 3], strided(x, "shifted"), x.transpose(0, 1).contiguous().transpose(0, 1)):
        assert all(torch.equal(a, c) for a, c in zip(want, sc.beam_select(y, scores.cuda(), n)))
    one = x[:, :1].expand(b, k, v)                       # stride 0
    check(one, scores, n)
    # flags as truth values; several streams at once, one given
    done = torch.rand((b, k), generator=g) < 0.5
    a = sc.beam_select(x, scores.cuda(), n, finished=done.cuda(), end_token=7)
    c = sc.beam_select(x, scores.cuda(), n, finished=done.to(torch.uint8).cuda(), end_token=7)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    dev_scores = scores.cuda()
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(sc.beam_select(x, dev_scores, n))
    outs.append(sc.beam_select(x, dev_scores, n, stream=streams[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in outs for p, q in zip(want, o))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_every_nan_is_masked(dt):
    # quiet and signalling ones of either sign, in the first, inner and last vectors, count for nothing
    v, bits = 2311, {"bf16": (torch.int16, 0x7f80, 0x40), "f16": (torch.int16, 0x7c00, 0x200),
                     "f32": (torch.int32, 0x7f800000, 0x400000)}[dt]
    kind, top, quiet = bits
    x = normal(gen(14), (2, 3, v), dt)
    masked = x.clone()
    sign = torch.iinfo(kind).min
    for i, at in enumerate((0, 1, 2, 700, 701, 1333, v - 2, v - 1)):
        nan = (top | (quiet if i % 2 else 1)) + (sign if i % 4 > 1 else 0)
        x.view(kind)[:, :, at] = nan
        masked[:, :, at] = -INF
    assert int(x.isnan().sum()) == 8 * 6
    s = -torch.rand((2, 3), generator=gen(15)).cuda()
    assert all(torch.equal(a, b) for a, b in zip(sc.beam_select(x, s, 16), sc.beam_select(masked, s, 16)))


def test_far_rows():
    # beams whose rows pass 2^32 bytes
    step = (1 << 30) + 5
    big = torch.zeros(2 * step + 4000, dtype=torch.bfloat16, device="cuda")
    x0 = normal(gen(12), (1, 3, 3999), "bf16")
    far = big.as_strided((1, 3, 3999), (3 * step, step, 1))
    far.copy_(x0)
    s = torch.zeros(1, 3, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(sc.beam_select(far, s, 16), sc.beam_select(x0, s, 16)))
    del big, far
    torch.cuda.empty_cache()


def test_largest_vocabulary():
    # places up to 2^31 - 2 in a row of 4 GiB; all but four logits are 0, which the first of them win
    v = 2 ** 31 - 1
    x = torch.zeros((1, 1, v), dtype=torch.bfloat16, device="cuda")
    great = {v - 1: 4.0, 0: 3.0, 5: 2.0, 2 ** 30 + 1: 1.0}
    for at, value in great.items():
        x[0, 0, at] = value
    got = sc.beam_select(x, torch.zeros(1, 1, device="cuda"), 6)
    assert got[2].tolist() == [list(great) + [1, 2]] and got[1].tolist() == [[0] * 6]
    lse = math.log(v - 4 + sum(math.exp(l) for l in great.values()))
    want = torch.tensor(list(great.values()) + [0.0, 0.0], dtype=torch.float64) - lse
    assert bool(((got[0][0].cpu().double() - want).abs() <= want.abs() * 2.0 ** -24 + 1e-9).all())
    del x
    torch.cuda.empty_cache()


def test_more_rows_than_a_launch_takes():
    # 2^22 workgroups a launch: the rows at its end and behind it
    b, k, v = 65540, 64, 3
    g = torch.Generator(device="cuda").manual_seed(13)
    x = torch.randn((b, k, v), generator=g, device="cuda").bfloat16()
    s = torch.randn((b, k), generator=g, device="cuda")
    got = sc.beam_select(x, s, 2)
    for lo, hi in ((0, 30000), (30000, b)):
        part = sc.beam_select(x[lo:hi], s[lo:hi].contiguous(), 2)
        assert all(torch.equal(a[lo:hi], c) for a, c in zip(got, part))
    full = s.double()[..., None] + torch.log_softmax(x.double(), -1)
    assert bool(((got[0][:, 0].double() - full.view(b, -1).max(-1).values).abs() < 1e-6).all())


# batch, beams, rows' shapes and types
REORDERS = [(1, 1, [((5,), "f32")]), (1, 4, [((3, 768), "bf16"), ((768, 16), "f32")]), (3, 2, [((), "i64"), ((1,), "u8")]),
            (2, 8, [((16,), "u8"), ((17,), "u8"), ((15,), "f16"), ((333, 3), "f32")]),
            (5, 5, [((1000,), "bf16"), ((0,), "f32"), ((4099,), "bf16")]), (2, 16, [((5000,), "f32")]),
            (1, 17, [((777,), "f16")]), (2, 32, [((130, 5), "f32"), ((3,), "u8")]), (2, 33, [((97,), "bf16")]),
            (1, 64, [((1025,), "f32"), ((7,), "i64")]), (300, 4, [((60,), "f32")])]
KINDS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i64": torch.int64, "u8": torch.uint8}


def states_of(g, b, k, rows):
    out = []
    for i, (shape, kind) in enumerate(rows):
        raw = torch.randint(0, 256, ((b * k,) + shape + (KINDS[kind].itemsize,)), generator=g, dtype=torch.uint8)
        t = raw.view(KINDS[kind]).squeeze(-1).view((b * k,) + shape)
        out.append((t.view((b, k) + shape) if i % 2 else t).cuda())
    return out


def raw(t, b, k):
    return t.contiguous().view(b, k, -1).view(torch.uint8).cpu().numpy() if t.numel() else np.zeros((b, k, 0), np.uint8)


@pytest.mark.parametrize("case", REORDERS, ids=[f"{c[0]}-{c[1]}-{len(c[2])}" for c in REORDERS])
@pytest.mark.parametrize("kind", ["any", "same", "first", "swap", "outside"])
def test_reorder(case, kind):
    b, k, rows = case
    g = gen(b * 100 + k)
    p = torch.randint(0, k, (b, k), generator=g)
    own = torch.arange(k).expand(b, k)
    if kind == "same":
        p = own.clone()
    elif kind == "first":
        p = torch.zeros_like(p)
    elif kind == "swap":
        p = own.flip(1).clone()
    elif kind == "outside":
        p = torch.where(torch.rand((b, k), generator=g) < 0.5, p, torch.tensor([-1, k, 2 ** 31 - 1, -2 ** 31])[p % 4])
    states = states_of(g, b, k, rows)
    want = [ref.reorder(raw(t, b, k), p.numpy()) for t in states]
    before = [t.clone() for t in states]
    fresh = [torch.full_like(t, 3) for t in states]
    got = sc.beam_reorder(states, p.int().cuda(), new_states=fresh)
    assert all(x is y for x, y in zip(got, fresh))
    for t, s, w in zip(got, states, want):
        assert np.array_equal(raw(t, b, k), w)
    for s, w in zip(states, before):
        assert torch.equal(s.view(torch.uint8) if s.numel() else s, w.view(torch.uint8) if w.numel() else w)
    moved = sc.beam_reorder(states, p.int().cuda())
    assert all(x is y for x, y in zip(moved, states))
    for t, w in zip(states, want):
        assert np.array_equal(raw(t, b, k), w)


def test_reorder_many_and_unaligned():
    g = gen(30)
    b, k = 2, 4
    p = torch.randint(0, k, (b, k), generator=g).int()
    big = torch.randint(0, 256, (150 * 400 + 1,), generator=g, dtype=torch.uint8).cuda()
    states = [big[1 + 400 * i:1 + 400 * i + b * k * (20 + i % 30)].view(b, k, 20 + i % 30) for i in range(150)]
    keep = big.clone()
    want = [ref.reorder(t.cpu().numpy(), p.numpy()) for t in states]
    sc.beam_reorder(states, p.cuda())
    for t, w in zip(states, want):
        assert np.array_equal(t.cpu().numpy(), w)
    # nothing beside them moved
    mask = torch.ones_like(big, dtype=torch.bool)
    for i in range(150):
        mask[1 + 400 * i:1 + 400 * i + b * k * (20 + i % 30)] = False
    assert torch.equal(big[mask], keep[mask])
    assert sc.beam_reorder([], p.cuda()) == []


def test_reorder_far():
    # rows of 2 GiB in two beams
    n = (1 << 31) + 24
    big = torch.zeros((1, 2, n), dtype=torch.uint8, device="cuda")
    big[0, 1, n - 20:], big[0, 1, :9] = 5, 6
    sc.beam_reorder([big], torch.tensor([[1, 1]], dtype=torch.int32, device="cuda"))
    assert int(big[0, 0, n - 20:].min()) == 5 and int(big[0, 0, :9].min()) == 6 and int(big[0, 0, 9:n - 20].max()) == 0
    del big
    torch.cuda.empty_cache()


def test_search_in_a_graph():
    # a step of beam search with recurrent states, captured once: gated scan step, logits, choice, states in
    # place.  Replayed with eager work between, against the same steps uncaptured
    b, k, d, v = 2, 4, 96, 1501
    g = gen(40)
    table = normal(g, (v, d), "bf16", 0.3)
    head = normal(g, (d, v), "bf16", 0.3)
    rate = torch.rand(d, generator=g).cuda()
    first_state = torch.randn((b * k, d), generator=g).cuda()
    end = 7

    def start():
        scores = torch.full((b, k), -INF, device="cuda")
        scores[:, 0] = 0
        return {"state": first_state.clone(), "scores": scores, "done": torch.zeros((b, k), dtype=torch.uint8, device="cuda"),
                "token": torch.ones((b, k), dtype=torch.int32, device="cuda"),
                "text": torch.zeros((b, k, 12), dtype=torch.int32, device="cuda"),
                "at": torch.zeros(1, dtype=torch.int64, device="cuda")}

    def step(s):
        e = sc.embedding(table, s["token"].view(-1), scale=3.0)
        y = sc.gated_scan_step(s["state"], e, e, rate)
        logits = (y @ head).view(b, k, v)
        scores, parents, tokens = sc.beam_select(logits, s["scores"], k, finished=s["done"], end_token=end)
        sc.beam_reorder([s["state"], s["text"], s["done"]], parents)
        s["scores"].copy_(scores)
        s["token"].copy_(tokens)
        s["done"].bitwise_or_((tokens == end).to(torch.uint8))
        s["text"].index_copy_(2, s["at"], tokens[..., None])
        s["at"].add_(1)
        return scores, parents, tokens

    eager = start()
    want = [[t.clone() for t in step(eager)] for _ in range(12)]
    held = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(start())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for n, t in start().items():
        held[n].copy_(t)
    for i in range(12):
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(out, want[i]):
            assert torch.equal(a, w), i
    for n in held:
        assert torch.equal(held[n], eager[n]), n
    # each step's best is what the oracle chooses from its logits
    assert bool((held["scores"][:, :-1] >= held["scores"][:, 1:]).all())


def test_refusals_leave_outputs():
    x, s = torch.randn(2, 3, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    for call in (lambda: sc.beam_select(x, s, 151), lambda: sc.beam_select(x, s, 4, out_scores=x[0, 0, :8].view(2, 4)),
                 lambda: sc.beam_select(x, s, 4, finished=s.to(torch.uint8), end_token=50),
                 lambda: sc.beam_select(x.cpu(), s, 4), lambda: sc.beam_select(x, s.cpu(), 4)):
        with pytest.raises((ValueError, NotImplementedError)):
            call()
    with pytest.raises(NotImplementedError):
        sc.beam_select(x, s, 65)
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    y = x.clone()
    with pytest.raises(ValueError):
        sc.beam_reorder([x, x], p)                       # moved twice
    with pytest.raises(ValueError):
        sc.beam_reorder([x.view(-1)[:240].view(2, 3, 40)], p, [x.view(-1)[1:241].view(2, 3, 40)])
    assert torch.equal(x, y)
