"""Oracle of the gated scan: the definition token by token in float64 numpy, with the
bounds of ``sequence_ref`` on what float32 arithmetic may add.

Beyond those: the kernels carry a state over a run of tokens by 2 to the sum of their
decays' logarithms, at most 40 of them added one after another (16 tokens, 8 waves, 16
chunks).  A logarithm's rounding and those of its sums move the decay by up to 4 EPS of
the logarithm, which is counted with each token's decay."""
import numpy as np

from sequence_ref import EPS, V, _live, _sig, sigmoid, silu, silu_slope, stack


def _neg(v):
    return V(-v.val, v.mag, v.err)


def gates(forget, rate):
    """Decay a, weight w, both sides of the gate, and with a rate p / w and p (V each)."""
    s, down = sigmoid(V(forget)), sigmoid(V(-forget))
    if rate is None:
        a = V(s.val, s.mag, s.err + 4 * EPS * np.abs(np.log(np.maximum(s.val, 1e-300))) * s.val)
        return a, down, s, down, None, None
    r = np.maximum(rate, 0.0)
    p = V(np.broadcast_to(r, s.val.shape)) * s
    m = V(-p.val, p.mag, p.err)
    a = m.func(np.exp, np.exp(-p.val))
    a.err = a.err + 4 * EPS * p.val * a.val
    # 1 - a^2 by a polynomial below p = 1/4, where it is good to 2 EPS and its five steps
    # to one each; above by the difference, which has a^2's error and one rounding
    a2 = np.exp(-2 * p.val)
    q = -np.expm1(-2 * p.val)
    far = 2 * a.val * a.err + 3 * EPS
    near = 2 * a2 * p.err + 7 * EPS * q
    err = np.where(p.val < 0.2, near, np.where(p.val > 0.3, far, np.maximum(near, far)))
    w = np.sqrt(q)
    safe = np.where(w > 0, w, 1.0)
    wv = V(w, w, np.where(w > 0, err / (2 * safe), 0.0) + 2 * EPS * w)
    pw = p.val / safe
    pv = V(pw, pw, np.where(w > 0, p.err / safe + pw * wv.err / safe, 0.0) + 3 * EPS * pw)
    return a, wv, s, down, pv, p


def gated(x, forget, rate=None, input_gate=None, z=None, initial=None, lengths=None, dy=None,
          dfinal=None, depth=None):
    """All arrays float64 numpy; returns a dict of V (y, state and, given dy, the gradients)."""
    b, l, d = x.shape
    on = np.stack([_live(lengths, b, t) for t in range(l)], 1)[..., None] if l else np.ones((b, 0, 1), bool)
    clean = lambda v: V(np.where(on, v, 0.0))  # noqa: E731
    xv = clean(x)
    a, w, s, down, pw, p = gates(clean(forget).val, rate)
    one = V(np.ones_like(x))
    v = one if input_gate is None else sigmoid(clean(input_gate))
    vdown = None if input_gate is None else sigmoid(V(-clean(input_gate).val))
    u = w * v * xv
    h = V(np.zeros((b, d))) if initial is None else V(initial.copy())
    hs = [h]
    for t in range(l):
        new = a[:, t] * h + u[:, t]
        k = on[:, t]
        h = V(np.where(k, new.val, h.val), np.where(k, new.mag, h.mag), np.where(k, new.err, h.err))
        hs.append(h)
    none = V(np.zeros((b, 0, d)))
    path = stack(hs[1:], 1) if l else none
    before = stack(hs[:-1], 1) if l else none
    zv = None if z is None else clean(z)
    out = {"y": (path if z is None else path * silu(zv)).where(on), "state": h}
    if dy is None:
        return out
    dyv = clean(dy)
    q = dyv if z is None else dyv * silu(zv)
    if z is not None:
        out["dz"] = (dyv * path * silu_slope(zv)).where(on)
    c = V(np.zeros((b, d))) if dfinal is None else V(dfinal.copy())
    gs = []
    for t in range(l - 1, -1, -1):
        g = q[:, t] + c
        move = a[:, t] * g
        k = on[:, t]
        gs.append(g.where(k))
        c = V(np.where(k, move.val, c.val), np.where(k, move.mag, c.mag), np.where(k, move.err, c.err))
    out["dstate"] = c
    g = stack(gs[::-1], 1) if l else none
    out["dx"] = (g * w * v).where(on)
    if input_gate is not None:
        out["dinput_gate"] = (g * w * v * xv * vdown).where(on)
    if rate is None:
        out["dforget"] = (g * (before + _neg(v * xv)) * s * down).where(on)
    else:
        E = (g * (v * xv * a * a * pw + _neg(p * a * before))).where(on)
        out["dforget"] = (E * down).where(on)
        # a wave adds its 8 tokens, 8 waves, then the chunks of 64 tokens of all sequences
        depth = 16 + b * (l // 64 + 1) if depth is None else depth
        total = E.sum(1, 1).sum(0, depth) if l else V(np.zeros(d))
        r = np.where(rate > 0, rate, 1.0)
        out["drate"] = (total * V(1 / r)).where(rate > 0)
    return out
