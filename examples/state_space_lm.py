"""A small state space language model on the library's sequence operators.

    python examples/state_space_lm.py [--steps 100] [--dtype bf16]

Embedding, causal convolution and selective scan make the model; it learns a rule that gives
each token from the one three places before (sequences padded to unequal lengths), forward and
backward through the library's kernels, and then answers token by token with the single-token steps, captured into one HIP
graph.  Prints the loss on the way, how far the steps' logits are from the whole sequence's,
and the share of tokens that the model continues right.
"""
import argparse
import math
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_amd as sc  # noqa: E402
from stream_compaction_amd import autograd as ops  # noqa: E402


class Layer(nn.Module):
    """norm, projection, convolution, scan with gate, projection, residual."""

    def __init__(self, model, inner, states, rank, width, dtype):
        super().__init__()
        self.states, self.rank = states, rank
        self.norm = nn.LayerNorm(model, dtype=dtype)
        self.enter = nn.Linear(model, 2 * inner, bias=False, dtype=dtype)
        self.select = nn.Linear(inner, rank + 2 * states, bias=False, dtype=dtype)
        self.step_up = nn.Linear(rank, inner, bias=False, dtype=dtype)
        self.leave = nn.Linear(inner, model, bias=False, dtype=dtype)
        self.filter = nn.Parameter((torch.rand(inner, width) * 2 - 1) / math.sqrt(width))
        self.filter_bias = nn.Parameter(torch.zeros(inner))
        self.log_A = nn.Parameter(torch.arange(1, states + 1).float().log().repeat(inner, 1))
        self.D = nn.Parameter(torch.ones(inner))
        target = torch.exp(torch.rand(inner) * math.log(100.0) + math.log(0.001))
        self.dt_bias = nn.Parameter(torch.log(torch.expm1(target)))

    def _selected(self, c):
        """Step, B and C of each token; B and C are views into one projection."""
        low, B, C = self.select(c).split([self.rank, self.states, self.states], -1)
        return self.step_up(low), B.unsqueeze(-2), C.unsqueeze(-2)

    def forward(self, u, lengths=None):
        """``[batch, length, model]`` to the same, and the state that steps go on from."""
        x, z = self.enter(self.norm(u)).chunk(2, -1)
        c, window = ops.causal_conv(x, self.filter, self.filter_bias, lengths=lengths)
        dt, B, C = self._selected(c)
        y, state = ops.selective_scan(c, dt, -self.log_A.exp(), B, C, self.D, z, self.dt_bias,
                                      softplus=True, lengths=lengths)
        return u + self.leave(y), (window, state)

    def step(self, u, cache):
        """One token, ``[batch, model]``; the cache moves on in place."""
        window, state = cache
        x, z = self.enter(self.norm(u)).chunk(2, -1)
        c = sc.causal_conv_step(window, x, self.filter, self.filter_bias)
        dt, B, C = self._selected(c)
        y = sc.selective_scan_step(state, c, dt, -self.log_A.exp(), B, C, self.D, z, self.dt_bias,
                                   softplus=True)
        return u + self.leave(y)


class Model(nn.Module):
    def __init__(self, vocabulary, model=64, inner=128, states=16, rank=8, width=4, layers=2,
                 dtype=torch.float32):
        super().__init__()
        self.table = nn.Parameter((torch.randn(vocabulary, model) / math.sqrt(model)).to(dtype))
        self.scale = math.sqrt(model)
        self.layers = nn.ModuleList(Layer(model, inner, states, rank, width, dtype)
                                    for _ in range(layers))
        self.norm = nn.LayerNorm(model, dtype=dtype)

    def forward(self, ids, lengths=None):
        u, cache = ops.embedding(self.table, ids, self.scale), []
        for layer in self.layers:
            u, c = layer(u, lengths)
            cache.append(c)
        return self.norm(u) @ self.table.t(), cache

    def step(self, ids, cache):
        u = sc.embedding(self.table, ids, self.scale)
        for layer, c in zip(self.layers, cache):
            u = layer.step(u, c)
        return self.norm(u) @ self.table.t()


LAG = 3


def sequences(gen, rule, size, length):
    """Token sequences that follow ``rule``, ``ids[t] = rule[ids[t - LAG]]``."""
    ids = torch.randint(0, rule.numel(), (size, LAG), generator=gen)
    while ids.shape[1] < length:
        ids = torch.cat([ids, rule[ids[:, -LAG:]]], 1)
    return ids[:, :length]


def train(model, steps, gen, rule, length=48, size=32):
    """Mean loss of the first and of the last five steps."""
    optimizer = torch.optim.AdamW(model.parameters(), lr=1e-2, weight_decay=0.01)
    losses = []
    for i in range(steps):
        ids = sequences(gen, rule, size, length)
        lengths = torch.randint(length // 2, length + 1, (size,), generator=gen)
        # padding is a masked token
        ids = torch.where(torch.arange(length) < lengths[:, None], ids, torch.full_like(ids, -1)).cuda()
        logits, _ = model(ids, lengths.int().cuda())
        loss = nn.functional.cross_entropy(logits[:, LAG - 1:-1].flatten(0, 1).float(),
                                           ids[:, LAG:].flatten(), ignore_index=-1)
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
        if i % 20 == 0 or i + 1 == steps:
            print(f"step {i}: loss {float(losses[-1]):.3f}", flush=True)
    values = torch.stack(losses).tolist()
    return sum(values[:5]) / len(values[:5]), sum(values[-5:]) / len(values[-5:])


@torch.no_grad()
def answer(model, prompt, count):
    """Greedy continuation of ``prompt`` (all of one length), one captured step per token:
    the tokens and the logits that gave them."""
    logits, cache = model(prompt)
    token = logits[:, -1].argmax(-1)
    tokens, seen = [token.clone()], []
    warm = [(w.clone(), s.clone()) for w, s in cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.step(token, warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model.step(token, cache)
        best = out.argmax(-1)
    for _ in range(count - 1):
        graph.replay()
        seen.append(out.clone())
        token.copy_(best)
        tokens.append(token.clone())
    return torch.stack(tokens, 1), torch.stack(seen, 1)


def run(steps=100, dtype="f32", vocabulary=32, seed=0):
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    kind = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    model = Model(vocabulary, dtype=kind).cuda()
    rule = torch.randperm(vocabulary, generator=gen)
    first, last = train(model, steps, gen, rule)
    whole = sequences(gen, rule, 16, 48).cuda()
    prompt = whole[:, :21].contiguous()
    tokens, seen = answer(model, prompt, 20)
    with torch.no_grad():
        again, _ = model(torch.cat([prompt, tokens[:, :-1]], 1))
    off = float((again[:, prompt.shape[1]:].float() - seen.float()).abs().max())
    span = float(again.float().abs().max())
    right = float((tokens == whole[:, prompt.shape[1]:prompt.shape[1] + 20]).float().mean())
    print(f"loss {first:.3f} -> {last:.3f}; steps' logits off by {off:.2e} of {span:.1f}; "
          f"{100 * right:.0f}% of tokens continued right", flush=True)
    return {"first": first, "last": last, "off": off, "span": span, "right": right}


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=100)
    parser.add_argument("--dtype", choices=("f32", "f16", "bf16"), default="f32")
    args = parser.parse_args()
    run(args.steps, args.dtype)
