"""The sequence operators at their edges on the GPU: batches that go out as several launches,
states whose decay over a chunk leaves float32's range, and infinities among the inputs."""
import pytest
import torch

import stream_compaction_amd as sc
from stream_compaction_amd.sequence import _scan_args
from test_gpu_sequence import act, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [13, 16])
def test_scan_step_over_several_launches(n):
    # a launch takes 2^21 workgroups of 256 lanes: here an odd number of sequences (299593),
    # two to a lane; the sequences at its end move once, in place as into a new state
    d = {13: 112, 16: 385}[n]
    lanes = d * (16 if n == 13 else 4)
    step = (1 << 21) // ((lanes + 255) // 256)
    b = step + 2
    assert step % 2 == 1
    r = torch.Generator(device="cuda").manual_seed(n)
    one = lambda *shape: torch.randn(shape, generator=r, device="cuda")  # noqa: E731
    x, dt = (one(1, d).bfloat16().expand(b, d) for _ in range(2))
    B, C = (one(b, 1, n).bfloat16() for _ in range(2))
    A, D = -torch.rand((d, n), generator=r, device="cuda"), one(d)
    state = one(1, d, n).expand(b, d, n).contiguous()
    first = state[0].clone()
    fresh = torch.empty_like(state)
    y = sc.selective_scan_step(state, x, dt, A, B, C, D, softplus=True, new_state=fresh)
    y2 = sc.selective_scan_step(state, x, dt, A, B, C, D, softplus=True)
    assert torch.equal(y, y2) and torch.equal(state, fresh)
    for i in (0, 1, step - 2, step - 1, step, step + 1):
        s = slice(i, i + 1)
        new = torch.empty((1, d, n), device="cuda")
        v = sc.selective_scan_step(first[None].clone(), x[s], dt[s], A, B[s], C[s], D,
                                   softplus=True, new_state=new)
        assert torch.equal(v, y[s]) and torch.equal(new[0], state[i]), f"sequence {i}"
    del state, fresh
    torch.cuda.empty_cache()


def whole(x, dt, A, B, C, **more):
    """``selective_scan`` in one piece, whatever its length."""
    k = {"D": None, "z": None, "dt_bias": None, "softplus": False, "initial_state": None,
         "lengths": None, **more}
    a = _scan_args(x, dt, A, B, C, k["D"], k["z"], k["dt_bias"], k["softplus"], k["initial_state"],
                   k["lengths"], False)
    y, state = torch.empty_like(x), torch.empty((a.batch, a.channels, a.states), device="cuda")
    sc.check(sc.lib().selective_scan(a, y.data_ptr(), state.data_ptr(), None,
                                     torch.cuda.current_stream().cuda_stream))
    return y, state


@pytest.mark.parametrize("n,signs", [(16, "A"), (13, "dt"), (40, "A")])
def test_growing_system_in_chunks(n, signs):
    # the decay over a chunk overflows, no state does: they are zero until the last tokens.  The
    # gradient likewise, from the other end
    b, l, d = 1, 1024, 20
    r = gen(300 + n)
    x, B, C = (act(r, s, "f32")[0] for s in ((b, l, d), (b, l, 1, n), (b, l, 1, n)))
    A = torch.rand((d, n), generator=r).cuda() + 0.5
    dt = torch.rand((b, l, d), generator=r).cuda() + 0.5
    if signs == "dt":
        A, dt = -A, -dt
    late = x.clone()
    late[:, :l - 20] = 0
    assert sc.lib().selective_scan_split_scratch_bytes(
        _scan_args(x, dt, A, B, C, None, None, None, False, None, None, False)) > 0
    y, state, starts = sc.selective_scan(late, dt, A, B, C, keep_starts=True)
    y1, state1 = whole(late, dt, A, B, C)
    assert bool(torch.isfinite(y1).all()) and bool(torch.isfinite(state1).all())
    # nothing is carried from chunk to chunk
    assert torch.equal(y, y1) and torch.equal(state, state1)
    # dy in the first 20 tokens alone: nothing is carried to them
    dy = act(r, (b, l, d), "f32")[0]
    dy[:, 20:] = 0
    zero = torch.zeros_like(x)
    _, _, starts = sc.selective_scan(zero, dt, A, B, C, keep_starts=True)
    g = sc.selective_scan_grad(dy, zero, dt, A, B, C, starts)
    # the same 64 tokens alone
    cut = lambda t: t[:, :64].contiguous()  # noqa: E731
    k = [cut(t) for t in (zero, dt)] + [A] + [cut(t) for t in (B, C)]
    _, _, s1 = sc.selective_scan(*k, keep_starts=True)
    g1 = sc.selective_scan_grad(cut(dy), *k, s1)
    for name in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(cut(g[name]), g1[name]), name
        assert not bool(g[name][:, 64:].any()), name
    assert torch.equal(g["dstate"], g1["dstate"]) and bool(torch.isfinite(g["dA"]).all())


def test_carried_state_past_the_factors_range():
    # a chunk's decay is below float32's least (2^-126) or above its greatest, the product with
    # the state is not; and an infinite state stays infinite
    b, l, d, n = 1, 1024, 16, 16
    A = torch.full((d, n), -1.0, device="cuda")
    zero = torch.zeros((b, l, d), device="cuda")
    B = torch.ones((b, l, 1, n), device="cuda")
    for per, start in ((0.6875, 2.0 ** 125), (-0.6875, 2.0 ** -125), (0.6875, float("inf"))):
        dt = torch.full((b, l, d), per, device="cuda")
        init = torch.full((b, d, n), start, device="cuda")
        y, state = sc.selective_scan(zero, dt, A, B, B, initial_state=init)
        y1, state1 = whole(zero, dt, A, B, B, initial_state=init)
        assert torch.equal(torch.isinf(y), torch.isinf(y1)) and not bool(torch.isnan(y).any())
        # token by token and in chunks: one rounding a token at most, and those of the exponents
        ok = torch.isfinite(y1) & (y1.abs() > 2.0 ** -110)
        assert int(ok.sum()) > 100 * d or start == float("inf")
        rel = ((y - y1).abs() / y1.abs())[ok]
        assert ok.sum() == 0 or float(rel.max()) <= 4 * l * 2.0 ** -24 + 2 * 140 * 2.0 ** -23


@pytest.mark.parametrize("n", [1, 13, 16, 20, 33])
@pytest.mark.parametrize("what", ["x", "dt"])
@pytest.mark.parametrize("l", [70, 600])
def test_infinite_input(n, what, l):
    # an infinite input makes its channel's state and outputs infinite from there on, and nothing
    # else: with positive B, C and D there is no difference of infinities
    b, d = 1, 19
    r = gen(320 + n)
    x, dt = (torch.rand((b, l, d), generator=r).cuda() + 0.1 for _ in range(2))
    B, C = (torch.rand((b, l, 1, n), generator=r).cuda() + 0.1 for _ in range(2))
    A, D = -torch.rand((d, n), generator=r).cuda() * 0.1 - 0.01, torch.ones(d, device="cuda")
    y0, state0 = sc.selective_scan(x, dt, A, B, C, D)
    t, c = 37, 17
    {"x": x, "dt": dt}[what][0, t, c] = float("inf")
    y, state = sc.selective_scan(x, dt, A, B, C, D)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, t:, c] = True
    assert bool((y[hit] == float("inf")).all()) and torch.equal(y[~hit], y0[~hit])
    assert bool((state[0, c] == float("inf")).all())
    keep = torch.arange(d) != c
    assert torch.equal(state[:, keep], state0[:, keep])


@pytest.mark.parametrize("n", [1, 13, 16, 20, 33])
@pytest.mark.parametrize("l", [70, 600])
def test_infinite_step_in_the_gradient(n, l):
    # behind an infinite step nothing of the tokens before it is left: their gradients are those
    # of a zero gradient from there on, and finite; so are all other channels'
    b, d, t, c = 1, 19, 37, 17
    r = gen(340 + n)
    x, dt, dy = (torch.rand((b, l, d), generator=r).cuda() + 0.1 for _ in range(3))
    B, C = (torch.rand((b, l, 1, n), generator=r).cuda() + 0.1 for _ in range(2))
    A = -torch.rand((d, n), generator=r).cuda() * 0.1 - 0.01
    dt[0, t, c] = float("inf")
    _, _, starts = sc.selective_scan(x, dt, A, B, C, keep_starts=True)
    g = sc.selective_scan_grad(dy, x, dt, A, B, C, starts)
    dt[0, t, c] = 1.0
    dy[0, t:, c] = 0
    cut = lambda v: v[:, :t].contiguous()  # noqa: E731
    k = [cut(x), cut(dt), A, cut(B), cut(C)]
    _, _, s0 = sc.selective_scan(*k, keep_starts=True)
    g0 = sc.selective_scan_grad(cut(dy), *k, s0)
    for name in ("dx", "ddt"):
        # sums over a state's own tokens: the same but for where a block of 16 begins
        assert torch.allclose(g[name][0, :t, c], g0[name][0, :, c], rtol=1e-5, atol=0), name
    keep = torch.arange(d) != c
    assert bool(torch.isfinite(g["dx"][..., keep]).all() & torch.isfinite(g["ddt"][..., keep]).all())
    assert bool((g["dx"][0, t, c] == float("inf")).all())


def test_convolution_past_the_caches():
    # a batch whose output is stored past the caches against its sequences, whose are not
    b, l, d = 3, 2051, 4096
    assert b * l * d * 2 >= 32 << 20 > l * d * 2
    r = gen(360)
    x = torch.randn(b, l, 2 * d, generator=r).bfloat16().cuda()[..., d:]
    w, bias = torch.randn(d, 4, generator=r).cuda(), torch.randn(d, generator=r).cuda()
    lengths = torch.tensor([l, 1000, 0], dtype=torch.int32).cuda()
    y, state = sc.causal_conv(x, w, bias, lengths=lengths)
    for i in range(b):
        one, last = sc.causal_conv(x[i:i + 1], w, bias, lengths=lengths[i:i + 1])
        assert torch.equal(one, y[i:i + 1]) and torch.equal(last, state[i:i + 1])
