"""The gated scan and beam search where they are used together: under torch's automatic differentiation
in a captured graph, and in the example model, which trains on padded sequences and searches for its
answers."""
import math
import os
import sys

import pytest
import torch
from torch.nn import functional as fn

from stream_compaction_amd import autograd as ops
from test_gpu_sequence import TYPES, act, gen

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import state_space_lm as lm  # noqa: E402

pytestmark = pytest.mark.gpu


def test_backward_in_a_graph():
    # forward and backward captured together, replayed on new inputs, with eager work of other leaves between
    r = gen(290)
    d, shape = 34, (2, 300)
    x, f, i, z, dy = (act(r, shape + (d,), "bf16")[0] for _ in range(5))
    first = [torch.rand(d, generator=r).cuda(), torch.randn((2, d), generator=r).cuda()]
    lengths = torch.tensor([300, 131], dtype=torch.int32, device="cuda")

    def work(leaves):
        rate, init = leaves
        y, state = ops.gated_scan(x, f, rate, i, z, init, lengths)
        return [y, state] + list(torch.autograd.grad([y, state], leaves, [dy, torch.ones_like(state)]))

    captured = [t.clone().requires_grad_(True) for t in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(captured)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(captured)
    eager = [t.clone().requires_grad_(True) for t in first]
    for n in range(3):
        for t in (x, f, i, z, dy):
            t.copy_(torch.randn(t.shape, generator=r))
        want = [t.detach().clone() for t in work(eager)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"replay {n}, output {j}"


def plain_layer(layer, u, lengths):
    """The example's gated layer in elementary torch operations, in u's type."""
    p = {n: t.to(u.dtype) for n, t in layer.named_parameters()}
    x, z = (fn.layer_norm(u, u.shape[-1:], p["norm.weight"], p["norm.bias"]) @ p["enter.weight"].t()).chunk(2, -1)
    width = p["filter"].shape[1]
    line = fn.pad(x, (0, 0, width - 1, 0))
    pre = p["filter_bias"] + sum(line[:, k:k + u.shape[1]] * p["filter"][:, k] for k in range(width))
    c = fn.silu(pre)
    forget, gate = (c @ p["gates.weight"].t() + p["gates.bias"]).chunk(2, -1)
    decay = torch.exp(p["log_rate"]) * torch.sigmoid(forget)
    a, w = torch.exp(-decay), torch.sqrt(-torch.expm1(-2 * decay))
    h, ys = torch.zeros_like(c[:, 0]), []
    for t in range(u.shape[1]):
        h = a[:, t] * h + (w * torch.sigmoid(gate) * c)[:, t]
        ys.append(h * fn.silu(z[:, t]))
    on = (torch.arange(u.shape[1], device=u.device) < lengths[:, None])[..., None]
    return u + torch.where(on, torch.stack(ys, 1), 0.0) @ p["leave.weight"].t()


def test_example_gradients():
    # the model's parameters against the same model in float64
    torch.manual_seed(3)
    model = lm.Model(19, model=24, inner=40, layers=2, mixer="gated").cuda()
    ids = torch.randint(0, 19, (3, 33), device="cuda")
    lengths = torch.tensor([33, 20, 7], dtype=torch.int32, device="cuda")
    on = torch.arange(33, device="cuda") < lengths[:, None]
    weight = torch.randn(3, 33, 19, device="cuda", dtype=torch.float64) * on[..., None]
    logits, _ = model(torch.where(on, ids, -1), lengths)
    (logits.double() * weight).sum().backward()
    got = {n: t.grad.double() for n, t in model.named_parameters()}
    wide = {n: t.detach().double().requires_grad_() for n, t in model.named_parameters()}
    u = torch.where(on[..., None], wide["table"][ids] * model.scale, 0.0)
    for i, layer in enumerate(model.layers):
        class View:
            def named_parameters(self, i=i):
                start = f"layers.{i}."
                return [(n[len(start):], t) for n, t in wide.items() if n.startswith(start)]
        u = plain_layer(View(), u, lengths)
    out = fn.layer_norm(u, u.shape[-1:], wide["norm.weight"], wide["norm.bias"]) @ wide["table"].t()
    (out * weight).sum().backward()
    # sums of some 60 tokens x 40 channels, whose terms cancel to about their root, through some 20 roundings
    # of 2^-24 each and the library's products: 60 x 40 x 20 x 2^-24 of the largest gradient at most
    for n, t in wide.items():
        off = float((got[n] - t.grad).abs().max())
        assert off <= 60 * 40 * 20 * 2.0 ** -24 * max(float(t.grad.abs().max()), 1.0), (n, off)


@pytest.mark.parametrize("mixer,dtype,beams", [("gated", "f32", 4), ("gated", "bf16", 3), ("selective", "f32", 5)])
def test_example_searches(mixer, dtype, beams):
    r = lm.run(steps=10, dtype=dtype, mixer=mixer, beams=beams)
    # steps and whole sequences round at different places: some steps of the type, a few layers
    room = 64 * float(torch.finfo(TYPES[dtype]).eps) * r["span"]
    assert math.isfinite(r["last"]) and r["off"] <= room
    # twenty tokens' log probabilities, each off by a logit's and a sum's rounding
    assert r["search_off"] <= 20 * 2 * room


def test_search_against_all_answers():
    # against all answers of three tokens: none better than the best, each with its own score, none twice
    torch.manual_seed(5)
    model = lm.Model(5, model=16, inner=24, layers=1, mixer="gated").cuda()
    prompt = torch.randint(0, 5, (3, 6), device="cuda")
    text, scores = lm.search(model, prompt, 3, 5)
    every = torch.cartesian_prod(*[torch.arange(5, device="cuda")] * 3)
    whole = torch.cat([prompt.repeat_interleave(125, 0), every.repeat(3, 1)], 1)
    with torch.no_grad():
        logits, _ = model(whole[:, :-1].contiguous())
    each = torch.log_softmax(logits[:, 5:].double(), -1).gather(-1, whole[:, 6:, None]).sum((1, 2)).view(3, 125)
    best = each.max(1).values
    assert bool((scores[:, 0].double() <= best + 1e-4).all())
    # and every answer that comes back has the score of its text
    at = (text[..., 0] * 25 + text[..., 1] * 5 + text[..., 2]).long()
    assert bool((each.gather(1, at) - scores.double()).abs().max() < 1e-4)
    assert bool((at.sort(1).values.diff(dim=1) > 0).all())
