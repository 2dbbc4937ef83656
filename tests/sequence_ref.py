"""Oracle of the sequence operators: the definitions token by token in float64
numpy, carrying with every value a bound of what float32 arithmetic may add.

A ``V`` holds a value, its magnitude (the same expression over absolute
values) and an absolute error bound.  One elementary operation costs ``EPS``
of the magnitude.  EPS is 4 float32 half steps: the kernels regroup the
recurrence (maps are composed before they are applied, so a product or sum of
the definition can stand for up to three of theirs) and use the hardware's
exponential and reciprocal, which are good to one step, two half steps.
"""
import numpy as np

EPS = 4 * 2.0 ** -24
# half a step of the output type, relative, and half its smallest step
HALF = {"f32": (2.0 ** -24, 2.0 ** -150), "f16": (2.0 ** -11, 2.0 ** -25),
        "bf16": (2.0 ** -8, 2.0 ** -134)}


class V:
    __slots__ = ("val", "mag", "err")

    def __init__(self, val, mag=None, err=None):
        self.val = np.asarray(val, np.float64)
        self.mag = np.abs(self.val) if mag is None else mag
        self.err = np.zeros_like(self.val) if err is None else err

    def __add__(self, o):
        o = o if isinstance(o, V) else V(o)
        mag = self.mag + o.mag
        return V(self.val + o.val, mag, self.err + o.err + EPS * mag)

    def __mul__(self, o):
        o = o if isinstance(o, V) else V(o)
        mag = self.mag * o.mag
        return V(self.val * o.val, mag, self.err * o.mag + self.mag * o.err + EPS * mag)

    def __getitem__(self, i):
        return V(self.val[i], self.mag[i], self.err[i])

    def func(self, f, slope):
        """f of this value, |f'| <= slope near it; the argument is first scaled by a
        constant (one rounding) and f costs two operations."""
        val = f(self.val)
        return V(val, np.abs(val), slope * (self.err + EPS * np.abs(self.val)) + 2 * EPS * np.abs(val))

    def sum(self, axis, depth=None):
        """Sum along an axis whose longest chain of additions is ``depth``."""
        n = self.val.shape[axis] if depth is None else depth
        mag = self.mag.sum(axis)
        return V(self.val.sum(axis), mag, self.err.sum(axis) + n * EPS * mag)

    def where(self, keep):
        return V(np.where(keep, self.val, 0.0), np.where(keep, self.mag, 0.0),
                 np.where(keep, self.err, 0.0))


def stack(vs, axis):
    return V(*(np.stack([getattr(v, n) for v in vs], axis) for n in ("val", "mag", "err")))



def _sig(v):
    return 1 / (1 + np.exp(-v))


def sigmoid(v):
    # sigmoid' <= sigmoid, so a relative change of the argument moves it by |v| of itself
    return v.func(_sig, _sig(v.val))


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    p = sigmoid(v)
    # s (1 + v (1 - s)): 1 - s loses the digits of s near 1, an error of EPS
    q = V(1 - p.val, np.abs(1 - p.val) + EPS, p.err + EPS)
    return p * (V(np.ones_like(p.val)) + v * q)


def softplus(v):
    # the derivative is the sigmoid; the series is about twelve operations
    r = v.func(lambda x: np.logaddexp(x, 0.0), _sig(v.val))
    r.err = r.err + 12 * EPS * r.mag
    return r


def _live(lengths, b, t):
    return np.ones(b, bool) if lengths is None else t < np.clip(lengths, 0, None)


def _spread(m, channels):
    """[batch, groups, states] to [batch, channels, states]."""
    return np.repeat(m, channels // m.shape[1], axis=1)


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, soft=False, initial=None, lengths=None,
         dy=None, dfinal=None, rows_depth=64):
    """All arrays float64 numpy; returns a dict of V (y, state and, given dy, the gradients)."""
    b, l, d = x.shape
    n = A.shape[1]
    g = B.shape[2]
    bias = 0.0 if dt_bias is None else dt_bias
    clean = lambda v, t: np.where(_live(lengths, b, t)[:, None], v[:, t], 0.0)  # noqa: E731
    zero = lambda: V(np.zeros((b, d, n)))  # noqa: E731
    h = zero() if initial is None else V(initial.copy())
    hs, steps, raws, decays, ys, sums = [h], [], [], [], [], []
    for t in range(l):
        on = _live(lengths, b, t)
        raw = V(clean(dt, t)) + V(np.broadcast_to(bias, (b, d)))
        s = softplus(raw) if soft else raw
        xt = V(clean(x, t))
        Bt = V(_spread(np.where(on[:, None, None], B[:, t], 0.0), d))
        Ct = V(_spread(np.where(on[:, None, None], C[:, t], 0.0), d))
        arg = V(s.val[..., None], s.mag[..., None], s.err[..., None]) * V(A[None])
        a = arg.func(np.exp, np.exp(arg.val))
        u = s * xt
        new = a * h + V(u.val[..., None], u.mag[..., None], u.err[..., None]) * Bt
        keep = on[:, None, None]
        h = V(np.where(keep, new.val, h.val), np.where(keep, new.mag, h.mag),
              np.where(keep, new.err, h.err))
        total = (Ct * h).sum(-1) + (V(np.zeros((b, d))) if D is None else V(D[None]) * xt)
        y = total if z is None else total * silu(V(clean(z, t)))
        ys.append(y.where(on[:, None]))
        hs.append(h)
        steps.append(s)
        raws.append(raw)
        decays.append(a)
        sums.append(total)
    none = V(np.zeros((b, 0, d)))
    out = {"y": stack(ys, 1) if l else none, "state": h}
    if dy is None:
        return out
    per = d // g
    acc = {k: [] for k in ("dx", "ddt", "dB", "dC", "dz")}
    dA, dD, db = [], [], []
    m = zero() if dfinal is None else V(dfinal.copy())
    for t in range(l - 1, -1, -1):
        on = _live(lengths, b, t)
        keep = on[:, None, None]
        xt, dyt = V(clean(x, t)), V(clean(dy, t))
        Bt = V(_spread(np.where(keep, B[:, t], 0.0), d))
        Ct = V(_spread(np.where(keep, C[:, t], 0.0), d))
        s, a = steps[t], decays[t]
        wide = lambda v: V(v.val[..., None], v.mag[..., None], v.err[..., None])  # noqa: E731
        if z is None:
            q = dyt
        else:
            zt = V(clean(z, t))
            q = dyt * silu(zt)
            acc["dz"].append((dyt * sums[t] * silu_slope(zt)).where(on[:, None]))
        G = (Ct * wide(q) + m).where(keep)
        acc["dC"].append((wide(q) * hs[t + 1]).where(keep))
        acc["dB"].append(G * wide(s * xt))
        gb = (G * Bt).sum(-1)
        move = a * G
        w = move * hs[t]
        ddt = gb * xt + (w * V(A[None])).sum(-1)
        acc["dx"].append((gb * s + (V(np.zeros((b, d))) if D is None else V(D[None]) * q)).where(on[:, None]))
        if soft:
            ddt = ddt * sigmoid(raws[t])
        ddt = ddt.where(on[:, None])
        acc["ddt"].append(ddt)
        db.append(ddt)
        dA.append(wide(s) * w)
        dD.append(q * xt)
        m = V(np.where(keep, move.val, m.val), np.where(keep, move.mag, m.mag),
              np.where(keep, move.err, m.err))
    out["dstate"] = m
    fold = lambda v: V(*(getattr(v, k).reshape(b, l, g, per, n) for k in ("val", "mag", "err"))).sum(3, min(per, rows_depth))  # noqa: E731
    for k, vs in acc.items():
        if k == "dz" and z is None:
            continue
        if not l:
            out[k] = V(np.zeros((b, 0, g, n) if k in ("dB", "dC") else (b, 0, d)))
            continue
        v = stack(vs[::-1], 1)
        out[k] = fold(v) if k in ("dB", "dC") else v
    # a lane adds its tokens, 64 lanes a tree, then block after block, sequence after sequence
    depth = 8 + 6 + l // 64 + 1 + b
    for k, vs, shape in (("dA", dA, (d, n)), ("dD", dD, (d,)), ("ddt_bias", db, (d,))):
        out[k] = stack(vs, 1).sum(1, depth).sum(0, 1) if l else V(np.zeros(shape))
    return out


def conv(x, w, bias=None, initial=None, lengths=None, act=True, dy=None, dfinal=None, depth=64):
    b, l, d = x.shape
    width = w.shape[1]
    out = {}
    y, fs, dx, ds = (np.zeros((b, l, d)), np.zeros((b, width - 1, d)), np.zeros((b, l, d)),
                     np.zeros((b, width - 1, d)))
    y, fs, dx, ds = V(y), V(fs), V(dx), V(ds)
    dw = V(np.zeros((b, d, width)))
    db = V(np.zeros((b, d)))
    for i in range(b):
        n = l if lengths is None else int(np.clip(lengths[i], 0, l))
        head = np.zeros((width - 1, d)) if initial is None else initial[i]
        line = V(np.concatenate([head, x[i, :n]], 0))
        pre = V(np.zeros((n, d))) if bias is None else V(np.broadcast_to(bias, (n, d)))
        for k in range(width):
            pre = pre + line[k:k + n] * V(w[:, k])
        r = silu(pre) if act else pre
        for name in ("val", "mag", "err"):
            getattr(y, name)[i, :n] = getattr(r, name)
            getattr(fs, name)[i] = getattr(line, name)[n:]
        if dy is None:
            continue
        g = V(dy[i, :n]) * silu_slope(pre) if act else V(dy[i, :n])
        back = V(np.zeros((n + width - 1, d)))
        if dfinal is not None:
            back.val[n:] += dfinal[i]
            back.mag[n:] += np.abs(dfinal[i])
        for k in range(width):
            part = g * V(w[:, k])
            for name in ("val", "mag", "err"):
                getattr(back, name)[k:k + n] += getattr(part, name)
            s = (g * line[k:k + n]).sum(0, depth)
            for name in ("val", "mag", "err"):
                getattr(dw, name)[i, :, k] = getattr(s, name)
        back.err += (width + 1) * EPS * back.mag
        s = g.sum(0, depth)
        for name in ("val", "mag", "err"):
            getattr(db, name)[i] = getattr(s, name)
            getattr(dx, name)[i, :n] = getattr(back, name)[width - 1:]
            getattr(ds, name)[i] = getattr(back, name)[:width - 1]
    out["y"], out["state"] = y, fs
    if dy is not None:
        out.update(dx=dx, dstate=ds, dweight=dw.sum(0, 1), dbias=db.sum(0, 1))
    return out


def embedding(weight, ids, scale):
    rows = weight.shape[0]
    ok = (ids >= 0) & (ids < rows)
    r = V(weight[np.clip(ids, 0, rows - 1)]) * V(np.float64(scale))
    return r.where(ok[..., None])


def embedding_grad(dout, ids, rows, scale, depth):
    ok = (ids >= 0) & (ids < rows)
    val, mag = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1]))
    np.add.at(val, ids[ok], dout[ok])
    np.add.at(mag, ids[ok], np.abs(dout[ok]))
    return V(val, mag, depth * EPS * mag) * V(np.float64(scale))


def excess(got, want, dt):
    """How far beyond its bound the worst element of got (float64) is, as a share of the
    bound: 0 when all are inside; inf for a NaN or a wrong shape."""
    if got.shape != want.val.shape:
        return np.inf
    if got.size == 0:
        return 0.0
    rel, tiny = HALF[dt]
    bound = want.err + rel * (np.abs(want.val) + want.err) + tiny
    off = np.abs(got - want.val)
    worst = np.max(np.where(np.isfinite(off), off / bound, np.inf))
    return float(worst) if worst > 1 else 0.0
