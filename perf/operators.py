"""Cases of the sequence operators (causal convolution, selective scan, embedding) and their plain forms.

A case names the operator and its direction in ``op``; activations are ``[batch, length, channels]``,
parameters and states float32.  The plain forms compute in float32 with elementary torch operations and
round once at the end.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
GIANT = 4 * 4096 * 4096 * 16          # state updates (tokens x channels x states) of the largest scan


def listed():
    return [
        # a short chat turn through one layer of a small model: latency counts
        {"name": "scan_prompt_short", "op": "scan", "batch": 1, "length": 45, "channels": 768, "states": 16,
         "groups": 1, "dtype": "bf16", "ragged": False, "gate": True, "softplus": True},
        # one long prompt before its answer: a batch of one, so only channels and time are parallel
        {"name": "scan_prompt_long", "op": "scan", "batch": 1, "length": 8192, "channels": 4096, "states": 16,
         "groups": 1, "dtype": "bf16", "ragged": False, "gate": True, "softplus": True},
        # a full batch of prompts of a server: the largest forward
        {"name": "scan_prompt_batch", "op": "scan", "batch": 4, "length": 4096, "channels": 4096, "states": 16,
         "groups": 1, "dtype": "f16", "ragged": True, "gate": True, "softplus": True},
        # a training step of one layer, forward and gradient
        {"name": "scan_train", "op": "scan_train", "batch": 4, "length": 2048, "channels": 2048, "states": 16,
         "groups": 1, "dtype": "bf16", "ragged": False, "gate": True, "softplus": True},
        # training in float32 on padded sequences, odd sizes, two groups of B and C, no gate
        {"name": "scan_train_odd", "op": "scan_train", "batch": 3, "length": 777, "channels": 522, "states": 13,
         "groups": 2, "dtype": "f32", "ragged": True, "gate": False, "softplus": True},
        # one token for each of 128 running answers
        {"name": "scan_step", "op": "scan_step", "batch": 128, "length": 1, "channels": 4096, "states": 16,
         "groups": 1, "dtype": "bf16", "ragged": False, "gate": True, "softplus": True},
        # the convolution before the scan, for the server's batch of prompts
        {"name": "conv_prompt", "op": "conv", "batch": 4, "length": 4096, "channels": 4096, "width": 4,
         "dtype": "bf16", "ragged": True, "silu": True},
        # its gradient in training
        {"name": "conv_grad", "op": "conv_grad", "batch": 4, "length": 2048, "channels": 2048, "width": 4,
         "dtype": "bf16", "ragged": False, "silu": True},
        # one token for each running answer: latency counts
        {"name": "conv_step", "op": "conv_step", "batch": 128, "length": 1, "channels": 4096, "width": 4,
         "dtype": "bf16", "ragged": False, "silu": True},
        # the tokens of a training batch looked up
        {"name": "embed_lookup", "op": "embed", "tokens": 16384, "rows": 50000, "channels": 2048,
         "dtype": "bf16", "scale": 45.25, "wide_ids": True},
        # and the table's gradient, with the skew of a language's tokens
        {"name": "embed_grad", "op": "embed_grad", "tokens": 16384, "rows": 50000, "channels": 2048,
         "dtype": "bf16", "scale": 45.25, "wide_ids": True},
        # fine tuning a small model on a few sequences, odd row length
        {"name": "embed_grad_odd", "op": "embed_grad", "tokens": 1531, "rows": 32003, "channels": 333,
         "dtype": "f32", "scale": 1.0, "wide_ids": False},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "conv", "conv_grad", "conv_step",
                     "embed", "embed_grad", "embed_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("embed"):
        return {"op": op, "tokens": _spread(rng, 1, 16384), "rows": _spread(rng, 500, 50000),
                "channels": rng.choice([_spread(rng, 64, 2048), 8 * _spread(rng, 8, 256)]), "dtype": dtype,
                "scale": rng.choice([1.0, 45.25]), "wide_ids": rng.random() < 0.5}
    step = op.endswith("_step")
    batch = _spread(rng, 1, 128) if step else rng.choice([1, 1, 2, 3, 4, 7])
    groups = rng.choice([1, 1, 1, 2, 4])
    channels = rng.choice([64 * _spread(rng, 1, 64), _spread(rng, 60, 4096)]) // groups * groups
    case = {"op": op, "batch": batch, "length": 1, "channels": channels, "dtype": dtype,
            "ragged": not step and rng.random() < 0.5}
    if op.startswith("conv"):
        case.update(width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8)
        most = 4 * 4096 * 4096 // (batch * channels)
    else:
        case.update(states=rng.choice([16, 16, 16, 8, 13, 32]), groups=groups, gate=rng.random() < 0.7,
                    softplus=rng.random() < 0.8)
        most = GIANT // (batch * channels * case["states"])
        most //= 8 if op == "scan_train" else 1
    if not step:
        case["length"] = _spread(rng, 1, max(1, min(8192, most)))
    return case


def _lengths(case):
    """Tokens of each sequence: a padded batch has full, part and (from three on) empty rows."""
    batch, length = case["batch"], case["length"]
    if not case["ragged"]:
        return [length] * batch
    return [length] + [(length * (2 * batch - 2 * b - 1)) // (2 * batch) for b in range(1, batch - 1)] + \
        ([0] if batch > 2 else [max(1, length // 3)] if batch == 2 else [])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": dict(case)}
    if case["op"].startswith("embed"):
        n, rows, d = case["tokens"], case["rows"], case["channels"]
        # a language's tokens: frequency falls with the rank, and about one in fifty is masked (-1)
        ids = torch.exp(uniform(n) * math.log(rows + 1)).floor().long().clamp_(1, rows) - 1
        ids = torch.where(uniform(n) < 0.02, torch.full_like(ids, -1), ids)
        s["ids"] = ids if case["wide_ids"] else ids.int()
        if case["op"] == "embed":
            s["weight"] = (normal(rows, d) * 0.02).to(dtype)
        else:
            s["dout"] = (normal(n, d) * 0.01).to(dtype)
        return s
    b, l, d = case["batch"], case["length"], case["channels"]
    lens = _lengths(case)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"].startswith("conv"):
        w = case["width"]
        s["weight"] = (uniform(d, w) * 2 - 1) / math.sqrt(w)
        s["bias"] = (uniform(d) * 2 - 1) / math.sqrt(w)
        s["state"] = normal(b, w - 1, d).to(dtype)
        if case["op"] == "conv_step":
            s["x"] = normal(b, d).to(dtype)
            s["new_state"] = torch.empty_like(s["state"])
            return s
        # the projection before gives the convolution's input and the gate side by side
        s["x"] = normal(b, l, 2 * d).to(dtype)[..., :d]
        if case["op"] == "conv_grad":
            s["dy"] = normal(b, l, d).to(dtype)
        return s
    n, groups = case["states"], case["groups"]
    s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * torch.exp(0.2 * normal(d, n))
    # steps between 0.001 and 0.1, even over the logarithm, moved by each token
    target = torch.exp(uniform(d) * math.log(100.0) + math.log(0.001))
    s["D"] = 1 + 0.1 * normal(d)
    lead = (b,) if case["op"] == "scan_step" else (b, l)
    x = normal(*lead, d)
    s["x"] = (x * torch.sigmoid(x)).to(dtype)
    if case["softplus"]:
        s["dt"] = (0.5 * normal(*lead, d)).to(dtype)
        s["dt_bias"] = torch.log(torch.expm1(target))
    else:
        s["dt"] = (target * torch.exp(0.5 * normal(*lead, d))).to(dtype)
        s["dt_bias"] = None
    s["B"] = normal(*lead, groups, n).to(dtype)
    s["C"] = normal(*lead, groups, n).to(dtype)
    s["z"] = normal(*lead, d).to(dtype) if case["gate"] else None
    s["state"] = normal(b, d, n)
    if case["op"] == "scan_step":
        s["new_state"] = torch.empty_like(s["state"])
    if case["op"] == "scan_train":
        s["dy"] = normal(b, l, d).to(dtype)
    return s


def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _valid(s, length):
    """[batch, length, 1]: which tokens exist."""
    t = torch.arange(length, device="cuda")
    if s["lengths"] is None:
        return torch.ones(1, length, 1, dtype=torch.bool, device="cuda")
    return (t < s["lengths"][:, None])[..., None]


def _recurrence(a, b):
    """h[t] = a[t] h[t-1] + b[t] along axis 1, h before the first being zero, by doubling."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _wide(v, channels):
    """[..., groups, states] to [..., channels, states]."""
    return v.float().repeat_interleave(channels // v.shape[-2], dim=-2)


def _plain_scan(s, train):
    c = s["case"]
    l, d = c["length"], c["channels"]
    ok = _valid(s, l)
    x = torch.where(ok, s["x"].float(), 0.0)
    raw = s["dt"].float()
    raw = raw if s["dt_bias"] is None else raw + s["dt_bias"]
    dt = torch.where(ok, _softplus(raw) if c["softplus"] else raw, 0.0)
    bb = torch.where(ok[..., None], _wide(s["B"], d), 0.0)
    cc = torch.where(ok[..., None], _wide(s["C"], d), 0.0)
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * bb
    b[:, 0] += a[:, 0] * s["state"]
    h = _recurrence(a, b)
    del b
    total = (cc * h).sum(-1) + s["D"] * x
    z = None if s["z"] is None else torch.where(ok, s["z"].float(), 0.0)
    y = total if z is None else total * _silu(z)
    y = torch.where(ok, y, 0.0).to(s["x"].dtype)
    out = {"y": y, "state": h[:, -1].contiguous()}
    if not train:
        return out
    dtype = s["x"].dtype
    dy = torch.where(ok, s["dy"].float(), 0.0)
    q = dy if z is None else dy * _silu(z)
    if z is not None:
        out["dz"] = (dy * total * _dsilu(z)).to(dtype)
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    grad = _recurrence(later, (cc * q[..., None]).flip(1)).flip(1)
    del later, cc
    groups = c["groups"]
    out["dC"] = (q[..., None] * h).unflatten(2, (groups, -1)).sum(3).to(dtype)
    out["dB"] = (grad * (dt * x)[..., None]).unflatten(2, (groups, -1)).sum(3).to(dtype)
    du = (grad * bb).sum(-1)
    out["dx"] = (du * dt + s["D"] * q).to(dtype)
    moved = grad * a
    out["dstate"] = moved[:, 0].contiguous()
    moved = moved * torch.cat([s["state"][:, None], h[:, :-1]], 1)
    ddt = du * x + (moved * s["A"]).sum(-1)
    ddt = torch.where(ok, ddt * torch.sigmoid(raw) if c["softplus"] else ddt, 0.0)
    out["ddt"] = ddt.to(dtype)
    if s["dt_bias"] is not None:
        out["ddt_bias"] = ddt.sum((0, 1))
    out["dA"] = (moved * dt[..., None]).sum((0, 1))
    out["dD"] = (q * x).sum((0, 1))
    return out


def _plain_scan_step(s):
    c = s["case"]
    d = c["channels"]
    x = s["x"].float()
    raw = s["dt"].float()
    raw = raw if s["dt_bias"] is None else raw + s["dt_bias"]
    dt = _softplus(raw) if c["softplus"] else raw
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * x)[..., None] * _wide(s["B"], d)
    y = (h * _wide(s["C"], d)).sum(-1) + s["D"] * x
    y = y if s["z"] is None else y * _silu(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": h}


def _plain_conv(s):
    c = s["case"]
    l, w = c["length"], c["width"]
    ok = _valid(s, l)
    x = torch.where(ok, s["x"].float(), 0.0)
    line = torch.cat([s["state"].float(), x], 1)
    pre = (line.unfold(1, w, 1) * s["weight"]).sum(-1) + s["bias"]
    lens = torch.full((c["batch"],), l, device="cuda") if s["lengths"] is None else s["lengths"].long()
    at = lens[:, None] + torch.arange(w - 1, device="cuda")
    last = torch.gather(line, 1, at[..., None].expand(-1, -1, c["channels"]))
    return ok, line, pre, last


def _plain_conv_grad(s):
    c = s["case"]
    l, w = c["length"], c["width"]
    ok, line, pre, _ = _plain_conv(s)
    g = s["dy"].float() * _dsilu(pre) if c["silu"] else s["dy"].float()
    g = torch.where(ok, g, 0.0)
    dtype = s["x"].dtype
    out = {"dbias": g.sum((0, 1)), "dweight": (line.unfold(1, w, 1) * g[..., None]).sum((0, 1))}
    side = torch.zeros_like(g[:, :w - 1])
    spread = torch.cat([side, g, side], 1).unfold(1, w, 1)          # g[t - w + 1 .. t] beside input t
    dline = (spread * s["weight"].flip(1)).sum(-1)
    out["dx"] = torch.where(ok, dline[:, w - 1:], 0.0).to(dtype)
    out["dstate"] = dline[:, :w - 1].to(dtype)
    return out


def _plain_conv_step(s):
    line = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (line.float() * s["weight"].t()).sum(1) + s["bias"]
    y = _silu(pre) if s["case"]["silu"] else pre
    return {"y": y.to(s["x"].dtype), "state": line[:, 1:].contiguous()}


def _plain_embed(s):
    ids, weight = s["ids"].long(), s["weight"]
    ok = ((ids >= 0) & (ids < weight.shape[0]))[:, None]
    return torch.where(ok, weight[ids.clamp(0, weight.shape[0] - 1)].float() * s["case"]["scale"], 0.0).to(weight.dtype)


def _plain_embed_grad(s):
    c = s["case"]
    ids = s["ids"].long()
    ok = ((ids >= 0) & (ids < c["rows"]))[:, None]
    part = torch.where(ok, s["dout"].float(), 0.0)
    total = torch.zeros(c["rows"], c["channels"], device="cuda")
    total.index_add_(0, ids.clamp(0, c["rows"] - 1), part)
    return (total * c["scale"]).to(s["dout"].dtype)


def _own(s):
    import stream_compaction_amd as sc
    c = s["case"]
    op = c["op"]
    if op == "embed":
        return sc.embedding(s["weight"], s["ids"], scale=c["scale"])
    if op == "embed_grad":
        return sc.embedding_grad(s["dout"], s["ids"], c["rows"], scale=c["scale"])
    if op == "conv":
        y, state = sc.causal_conv(s["x"], s["weight"], s["bias"], initial_state=s["state"],
                                  lengths=s["lengths"], silu=c["silu"])
        return {"y": y, "state": state}
    if op == "conv_grad":
        return sc.causal_conv_grad(s["dy"], s["x"], s["weight"], s["bias"], initial_state=s["state"],
                                   lengths=s["lengths"], silu=c["silu"])
    if op == "conv_step":
        y = sc.causal_conv_step(s["state"], s["x"], s["weight"], s["bias"], silu=c["silu"],
                                new_state=s["new_state"])
        return {"y": y, "state": s["new_state"]}
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "softplus": c["softplus"]}
    if op == "scan_step":
        y = sc.selective_scan_step(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"],
                                   new_state=s["new_state"], **more)
        return {"y": y, "state": s["new_state"]}
    if op == "scan":
        y, state = sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], initial_state=s["state"],
                                     lengths=s["lengths"], **more)
        return {"y": y, "state": state}
    y, state, starts = sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], initial_state=s["state"],
                                         lengths=s["lengths"], keep_starts=True, **more)
    grads = sc.selective_scan_grad(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], starts,
                                   lengths=s["lengths"], **more)
    return {"y": y, "state": state, **{k: v for k, v in grads.items() if v is not None}}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "embed":
        return _plain_embed(state)
    if op == "embed_grad":
        return _plain_embed_grad(state)
    if op == "conv":
        ok, _, pre, last = _plain_conv(state)
        y = torch.where(ok, _silu(pre) if state["case"]["silu"] else pre, 0.0)
        return {"y": y.to(state["x"].dtype), "state": last.to(state["x"].dtype)}
    if op == "conv_grad":
        return _plain_conv_grad(state)
    if op == "conv_step":
        return _plain_conv_step(state)
    if op == "scan_step":
        return _plain_scan_step(state)
    return _plain_scan(state, op == "scan_train")


def work(case):
    e = _BYTES[case["dtype"]]
    op = case["op"]
    if op.startswith("embed"):
        n, rows, d = case["tokens"], case["rows"], case["channels"]
        ids = n * (8 if case["wide_ids"] else 4)
        if op == "embed":       # the rows that are looked up are read once each, at most the whole table
            return {"bytes": ids + min(n, rows) * d * e + n * d * e, "flops": n * d}
        return {"bytes": ids + n * d * e + rows * d * e, "flops": 2 * n * d}
    b, d = case["batch"], case["channels"]
    tokens = sum(_lengths(case))
    padded = b * case["length"]
    if op.startswith("conv"):
        w = case["width"]
        params = 4 * d * (w + 1)
        state = b * (w - 1) * d * e
        if op == "conv_grad":
            return {"bytes": e * d * (2 * tokens + padded) + 2 * params + 2 * state, "flops": (6 * w + 8) * tokens * d}
        return {"bytes": e * d * (tokens + padded) + params + 2 * state, "flops": (2 * w + 4) * tokens * d}
    n, groups = case["states"], case["groups"]
    gate = 1 if case["gate"] else 0
    params = 4 * d * (n + 2)
    state = 4 * b * d * n
    wide = 2 * groups * n * e
    total = e * d * ((2 + gate) * tokens + padded) + wide * tokens + params + 2 * state
    flops = 7 * tokens * d * n
    if op == "scan_train":
        total += e * d * ((3 + gate) * tokens + (2 + gate) * padded) + wide * (tokens + padded) + 2 * params + state
        flops += 22 * tokens * d * n
    return {"bytes": total, "flops": flops}


def exact(case, seed):
    """The definition in 64 bits, token by token."""
    s = prepare(case, seed)
    op = case["op"]

    def wide(v):
        return None if v is None else v.double()

    def silu(v):
        return v / (1 + torch.exp(-v))

    def slope(v):
        p = 1 / (1 + torch.exp(-v))
        return p + v * p * (1 - p)

    if op.startswith("embed"):
        ids = s["ids"].cpu().long()
        ok = torch.nonzero((ids >= 0) & (ids < case["rows"]))[:, 0]
        if op == "embed":
            out = torch.zeros(case["tokens"], case["channels"], dtype=torch.float64)
            out[ok] = s["weight"].cpu().double()[ids[ok]] * case["scale"]
            return out
        out = torch.zeros(case["rows"], case["channels"], dtype=torch.float64)
        out.index_add_(0, ids[ok], s["dout"].cpu().double()[ok] * case["scale"])
        return out
    lens = _lengths(case)
    b, l, d = case["batch"], case["length"], case["channels"]
    if op.startswith("conv"):
        w = case["width"]
        weight, bias = wide(s["weight"]), wide(s["bias"])
        if op == "conv_step":
            rows = torch.cat([wide(s["state"]), wide(s["x"])[:, None]], 1)
            pre = bias + sum(rows[:, k] * weight[:, k] for k in range(w))
            return {"y": silu(pre) if case["silu"] else pre, "state": rows[:, 1:]}
        y = torch.zeros(b, l, d, dtype=torch.float64, device="cuda")
        state = wide(s["state"]).clone()
        dx, dstate = torch.zeros_like(y), torch.zeros_like(state)
        dweight, dbias = torch.zeros_like(weight), torch.zeros_like(bias)
        for i, n in enumerate(lens):
            rows = torch.cat([wide(s["state"][i]), wide(s["x"][i, :n])], 0)
            pre = bias + sum(rows[k:k + n] * weight[:, k] for k in range(w))
            y[i, :n] = silu(pre) if case["silu"] else pre
            state[i] = rows[n:]
            if op == "conv_grad":
                g = wide(s["dy"][i, :n]) * (slope(pre) if case["silu"] else 1.0)
                back = torch.zeros_like(rows)
                for k in range(w):
                    back[k:k + n] += g * weight[:, k]
                    dweight[:, k] += (g * rows[k:k + n]).sum(0)
                dbias += g.sum(0)
                dx[i, :n], dstate[i] = back[w - 1:], back[:w - 1]
        if op == "conv":
            return {"y": y, "state": state}
        return {"dx": dx, "dstate": dstate, "dweight": dweight, "dbias": dbias}
    groups = case["groups"]
    A, D, z = wide(s["A"]), wide(s["D"]), wide(s["z"])
    x = wide(s["x"])
    raw = wide(s["dt"]) + (0.0 if s["dt_bias"] is None else wide(s["dt_bias"]))
    dt = torch.logaddexp(raw, torch.zeros_like(raw)) if case["softplus"] else raw
    per = d // groups
    take = torch.arange(d, device="cuda") // per
    if op == "scan_step":
        h = torch.exp(dt[..., None] * A) * wide(s["state"]) + (dt * x)[..., None] * wide(s["B"])[:, take]
        y = (h * wide(s["C"])[:, take]).sum(-1) + D * x
        return {"y": y if z is None else y * silu(z), "state": h}
    live = torch.tensor(lens, device="cuda")
    h = wide(s["state"]).clone()
    total = torch.zeros(b, l, d, dtype=torch.float64, device="cuda")
    kept = []
    for t in range(l):
        on = (t < live)[:, None, None]
        new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * wide(s["B"][:, t])[:, take]
        kept.append(h if op == "scan_train" else None)
        h = torch.where(on, new, h)
        total[:, t] = (h * wide(s["C"][:, t])[:, take]).sum(-1) + D * x[:, t]
    ok = (torch.arange(l, device="cuda") < live[:, None])[..., None]
    y = torch.where(ok, total if z is None else total * silu(z), 0.0)
    if op == "scan":
        return {"y": y, "state": h}
    dy = torch.where(ok, wide(s["dy"]), 0.0)
    q = dy if z is None else dy * silu(z)
    out = {"y": y, "state": h}
    if z is not None:
        out["dz"] = dy * total * slope(z)
    out["dx"], ddt = torch.zeros_like(x), torch.zeros_like(x)
    out["dB"] = torch.zeros(b, l, groups, case["states"], dtype=torch.float64, device="cuda")
    out["dC"] = torch.zeros_like(out["dB"])
    out["dA"] = torch.zeros_like(A)
    grad, after = torch.zeros_like(h), h
    for t in range(l - 1, -1, -1):
        on = (t < live)[:, None, None]
        Bt, Ct = wide(s["B"][:, t])[:, take], wide(s["C"][:, t])[:, take]
        now = grad + torch.where(on, Ct * q[:, t, :, None], 0.0)
        seen = torch.where(on, now, 0.0)
        out["dC"][:, t] = torch.where(on, after * q[:, t, :, None], 0.0).unflatten(1, (groups, per)).sum(2)
        out["dB"][:, t] = (seen * (dt[:, t] * x[:, t])[..., None]).unflatten(1, (groups, per)).sum(2)
        du = (seen * Bt).sum(-1)
        moved = torch.exp(dt[:, t, :, None] * A) * seen
        out["dx"][:, t] = du * dt[:, t] + D * q[:, t]
        ddt[:, t] = du * x[:, t] + (moved * kept[t] * A).sum(-1)
        out["dA"] += (moved * kept[t] * dt[:, t, :, None]).sum(0)
        grad = torch.where(on, moved, grad)
        after = kept[t]
    out["dstate"] = grad
    if case["softplus"]:
        ddt = ddt / (1 + torch.exp(-raw))
    out["ddt"] = torch.where(ok, ddt, 0.0)
    if s["dt_bias"] is not None:
        out["ddt_bias"] = out["ddt"].sum((0, 1))
    out["dD"] = (q * torch.where(ok, x, 0.0)).sum((0, 1))
    return out
