"""The oracle of the sequence operators against central differences of its own
forward pass in float64, and the refusals of their C ABI, which are decided on
the host (so all of this runs without a GPU; the pointers are fake addresses)."""
import ctypes

import numpy as np
import pytest

import sequence_ref as ref
import stream_compaction_amd as sc
from stream_compaction_amd._sequence_abi import ConvArgs, ScanArgs, ScanGrads

OK, EINVAL, ENOTSUP, EALIAS, ESCRATCH = 0, 1, 2, 3, 4
D = sc.DTYPE_CODES


def slopes(f, x, h=1e-5):
    """Central differences of the scalar f at every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * h)
    return g


def near(got, want):
    # differences are good to h^2 of the third derivative and 1e-16 / h of the value
    assert np.max(np.abs(got - want)) <= 1e-7 * max(1.0, np.max(np.abs(want)))


@pytest.mark.parametrize("soft,gate,lengths", [(True, True, None), (False, True, [3, 0]),
                                               (True, False, [1, 3])])
def test_scan_gradient_is_the_forward_slope(soft, gate, lengths):
    r = np.random.default_rng(3)
    b, l, d, n, g = 2, 3, 4, 3, 2
    k = {"x": r.normal(size=(b, l, d)), "dt": 0.3 * r.normal(size=(b, l, d)) + (0 if soft else 0.5),
         "A": -r.uniform(0.1, 2, (d, n)), "B": r.normal(size=(b, l, g, n)),
         "C": r.normal(size=(b, l, g, n)), "D": r.normal(size=d), "dt_bias": r.normal(size=d),
         "initial": r.normal(size=(b, d, n)), "z": r.normal(size=(b, l, d)) if gate else None}
    dy, df = r.normal(size=(b, l, d)), r.normal(size=(b, d, n))

    def total():
        o = ref.scan(**k, soft=soft, lengths=lengths)
        return float((o["y"].val * dy).sum() + (o["state"].val * df).sum())

    o = ref.scan(**k, soft=soft, lengths=lengths, dy=dy, dfinal=df)
    for name, grad in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"),
                       ("D", "dD"), ("dt_bias", "ddt_bias"), ("initial", "dstate"), ("z", "dz")):
        if k[name] is not None:
            near(o[grad].val, slopes(total, k[name]))


@pytest.mark.parametrize("act,lengths,width", [(True, None, 3), (False, [4, 0], 4), (True, [1, 3], 2)])
def test_conv_gradient_is_the_forward_slope(act, lengths, width):
    r = np.random.default_rng(4)
    b, l, d = 2, 4, 3
    x, w, bias = r.normal(size=(b, l, d)), r.normal(size=(d, width)), r.normal(size=d)
    init = r.normal(size=(b, width - 1, d))
    dy, df = r.normal(size=(b, l, d)), r.normal(size=(b, width - 1, d))

    def total():
        o = ref.conv(x, w, bias, init, lengths, act)
        return float((o["y"].val * dy).sum() + (o["state"].val * df).sum())

    o = ref.conv(x, w, bias, init, lengths, act, dy=dy, dfinal=df)
    for v, grad in ((x, "dx"), (w, "dweight"), (bias, "dbias"), (init, "dstate")):
        near(o[grad].val, slopes(total, v))


def test_embedding_gradient_is_the_forward_slope():
    r = np.random.default_rng(5)
    w, ids = r.normal(size=(5, 3)), np.array([1, 4, -1, 1, 5, 0])
    do = r.normal(size=(6, 3))
    g = ref.embedding_grad(do, ids, 5, 1.5, 3)
    near(g.val, slopes(lambda: float((ref.embedding(w, ids, 1.5).val * do).sum()), w))


def test_bounds_hold_for_float32():
    # the definition run in plain float32 stays inside the oracle's bounds, a planted error
    # does not
    r = np.random.default_rng(6)
    b, l, d, n = 1, 200, 3, 4
    x, dt = r.normal(size=(b, l, d)).astype(np.float32), r.uniform(0.01, 0.2, (b, l, d)).astype(np.float32)
    A = -r.uniform(0.1, 4, (d, n)).astype(np.float32)
    B, C = (r.normal(size=(b, l, 1, n)).astype(np.float32) for _ in range(2))
    f = lambda v: v.astype(np.float64)  # noqa: E731
    want = ref.scan(f(x), f(dt), f(A), f(B), f(C))["y"]
    h, ys = np.zeros((b, d, n), np.float32), []
    for t in range(l):
        h = np.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * B[:, t]
        ys.append((h * C[:, t]).sum(-1))
    y = np.stack(ys, 1)
    assert y.dtype == np.float32
    assert ref.excess(f(y), want, "f32") == 0.0
    y[0, 100, 1] *= 1 + 2e-4
    assert ref.excess(f(y), want, "f32") > 1


P = 0x10000000                     # fake device addresses, 256 MiB apart
S = [P * (i + 1) for i in range(20)]


def conv_args(**k):
    a = ConvArgs(x=S[0], weight=S[1], bias=S[2], initial_state=S[3], lengths=S[4], batch=2,
                 length=10, channels=16, width=4, silu=1, dtype=D["bf16"])
    a.x_stride[:] = (160, 16)
    for name, v in k.items():
        if name == "x_stride":
            a.x_stride[:] = v
        else:
            setattr(a, name, v)
    return a


def test_conv_refusals():
    L = sc.lib()

    def call(y=S[5], fs=S[6], **k):
        return L.causal_conv(conv_args(**k), y, fs, None)
    assert L.causal_conv(None, S[5], S[6], None) == EINVAL
    assert call(dtype=D["f64"]) == ENOTSUP and call(dtype=0) == ENOTSUP
    assert call(width=0) == ENOTSUP and call(width=9) == ENOTSUP
    assert call(silu=2) == EINVAL
    assert call(batch=-1) == EINVAL and call(length=-1) == EINVAL and call(length=1 << 31) == EINVAL
    assert call(channels=0) == EINVAL and call(channels=(1 << 22) + 1) == EINVAL
    assert call(x=None) == EINVAL and call(weight=None) == EINVAL and call(y=None) == EINVAL
    assert call(x=S[0] + 1) == EINVAL and call(weight=S[1] + 2) == EINVAL and call(lengths=S[4] + 2) == EINVAL
    assert call(x_stride=(-160, 16)) == EINVAL and call(x_stride=(160, -1)) == EINVAL
    assert call(x_stride=(1 << 62, 16)) == EINVAL and call(x_stride=(160, 1 << 62)) == EINVAL
    assert call(y=S[0]) == EALIAS and call(y=S[0] + 2 * (160 + 159)) == EALIAS
    assert call(y=S[1]) == EALIAS and call(y=S[4]) == EALIAS and call(fs=S[5] + 4) == EALIAS
    assert call(fs=S[3]) == EALIAS
    assert call(batch=0) == OK                               # a no-op that never launches


def test_conv_grad_refusals():
    L = sc.lib()
    need = L.causal_conv_grad_scratch_bytes(conv_args())
    assert need > 0 and L.causal_conv_grad_scratch_bytes(conv_args(width=9)) == 0
    stride = (ctypes.c_int64 * 2)(160, 16)

    def call(dy=S[5], st=stride, df=S[6], dx=S[7], dw=S[8], db=S[9], di=S[10], s=S[11], sb=need, **k):
        return L.causal_conv_grad(conv_args(**k), dy, st, df, dx, dw, db, di, s, sb, None)
    assert call(dy=None) == EINVAL and call(st=None) == EINVAL and call(dx=None) == EINVAL
    assert call(dw=None) == EINVAL and call(s=None) == EINVAL and call(s=S[11] + 8) == EINVAL
    assert call(st=(ctypes.c_int64 * 2)(-1, 16)) == EINVAL
    assert call(sb=need - 1) == ESCRATCH
    assert call(dx=S[5]) == EALIAS and call(dw=S[1]) == EALIAS and call(s=S[7]) == EALIAS
    assert call(db=S[8] + 4) == EALIAS and call(di=S[6]) == EALIAS
    assert call(dtype=D["i32"]) == ENOTSUP


def test_conv_step_refusals():
    L = sc.lib()

    def call(st=S[5], ns=S[6], y=S[7], **k):
        return L.causal_conv_step(conv_args(**k), st, ns, y, None)
    assert call(st=None) == EINVAL and call(ns=None) == EINVAL and call(y=None) == EINVAL
    assert call(st=S[6] + 2) == EALIAS                       # overlapping, not the same
    assert call(y=S[5]) == EALIAS and call(y=S[0]) == EALIAS
    assert call(batch=1 << 20, channels=1 << 20) == EINVAL
    assert call(width=9) == ENOTSUP and call(batch=0) == OK


def scan_args(**k):
    a = ScanArgs(x=S[0], dt=S[1], B=S[2], C=S[3], z=S[4], A=S[5], D=S[6], dt_bias=S[7],
                 initial_state=S[8], lengths=S[9], batch=2, length=10, channels=16, states=8,
                 groups=2, softplus=1, dtype=D["f32"])
    for name in ("x_stride", "dt_stride", "z_stride"):
        getattr(a, name)[:] = (160, 16)
    for name in ("B_stride", "C_stride"):
        getattr(a, name)[:] = (160, 16, 8)
    for name, v in k.items():
        if name.endswith("_stride"):
            getattr(a, name)[:] = v
        else:
            setattr(a, name, v)
    return a


def test_scan_refusals():
    L = sc.lib()

    def call(y=S[10], fs=S[11], st=S[12], **k):
        return L.selective_scan(scan_args(**k), y, fs, st, None)
    assert L.selective_scan(None, S[10], S[11], None, None) == EINVAL
    assert call(dtype=D["f64"]) == ENOTSUP and call(states=0) == ENOTSUP and call(states=65) == ENOTSUP
    assert call(softplus=2) == EINVAL and call(groups=3) == EINVAL and call(groups=0) == EINVAL
    assert call(batch=-1) == EINVAL and call(length=1 << 31) == EINVAL and call(channels=0) == EINVAL
    for name in ("x", "dt", "B", "C", "A"):
        assert call(**{name: None}) == EINVAL, name
    assert call(y=None) == EINVAL
    for name in ("x", "dt", "B", "C", "z", "A", "D", "dt_bias", "initial_state", "lengths"):
        assert call(**{name: S[15] + 2}) == EINVAL, name     # not aligned to its element
    assert call(z_stride=(160, -16)) == EINVAL and call(B_stride=(160, 16, -8)) == EINVAL
    assert call(C_stride=(1 << 61, 16, 8)) == EINVAL
    for i in range(10):
        assert call(y=S[i]) == EALIAS, i
    assert call(fs=S[8]) == EALIAS and call(fs=S[10] + 16) == EALIAS and call(st=S[11]) == EALIAS
    assert call(batch=0) == OK
    # the starts: one state before every block of 64 to 512 tokens
    assert L.selective_scan_starts_bytes(scan_args()) == 2 * 16 * 8 * 4
    assert L.selective_scan_starts_bytes(scan_args(length=0)) == 0
    assert L.selective_scan_starts_bytes(scan_args(groups=3)) == 0


def scan_grads(**k):
    g = ScanGrads(dy=S[10], dfinal=S[11], starts=S[12], dx=S[13], ddt=S[14], dB=S[15], dC=S[16],
                  dz=S[17], dA=S[18], dD=S[19], ddt_bias=S[19] + 4096, dinitial=S[19] + 8192)
    g.dy_stride[:] = (160, 16)
    for name, v in k.items():
        if name == "dy_stride":
            g.dy_stride[:] = v
        else:
            setattr(g, name, v)
    return g


def test_scan_grad_refusals():
    L = sc.lib()
    need = L.selective_scan_grad_scratch_bytes(scan_args())
    assert need > 0 and L.selective_scan_grad_scratch_bytes(scan_args(states=99)) == 0
    W = S[19] + 0x1000000

    def call(a=None, s=W, sb=need, **k):
        return L.selective_scan_grad(scan_args(**(a or {})), scan_grads(**k), s, sb, None)
    for name in ("dy", "starts", "dx", "ddt", "dB", "dC", "dA", "dz"):
        assert call(**{name: None}) == EINVAL, name
    assert call(a={"z": None}) == EINVAL                     # dz without z
    assert L.selective_scan_grad(scan_args(), None, W, need, None) == EINVAL
    assert call(dy_stride=(160, -16)) == EINVAL
    assert call(s=None) == EINVAL and call(s=W + 4) == EINVAL and call(sb=need - 1) == ESCRATCH
    assert call(dx=S[10]) == EALIAS and call(dA=S[5]) == EALIAS and call(dB=S[16] + 64) == EALIAS
    assert call(dinitial=S[11]) == EALIAS and call(s=S[18]) == EALIAS


def test_scan_step_refusals():
    L = sc.lib()

    def call(st=S[10], ns=S[11], y=S[12], **k):
        return L.selective_scan_step(scan_args(**k), st, ns, y, None)
    assert call(st=None) == EINVAL and call(ns=None) == EINVAL and call(y=None) == EINVAL
    assert call(st=S[11] + 16) == EALIAS and call(y=S[10]) == EALIAS and call(y=S[0]) == EALIAS
    assert call(batch=1 << 20, channels=1 << 20) == EINVAL
    assert call(states=65) == ENOTSUP and call(batch=0) == OK


def test_embedding_refusals():
    L = sc.lib()
    f32, i64 = D["f32"], D["i64"]

    def call(w=S[0], i=S[1], o=S[2], n=10, rows=7, d=16, st=16, ty=f32, it=i64):
        return L.embedding(w, i, o, n, rows, d, st, ty, it, 1.0, None)
    assert call(ty=D["f64"]) == ENOTSUP and call(it=f32) == ENOTSUP
    assert call(n=-1) == EINVAL and call(n=1 << 31) == EINVAL and call(rows=0) == EINVAL
    assert call(d=0) == EINVAL and call(st=-1) == EINVAL and call(st=1 << 60) == EINVAL
    assert call(w=None) == EINVAL and call(i=None) == EINVAL and call(o=None) == EINVAL
    assert call(i=S[1] + 4) == EINVAL and call(o=S[2] + 2) == EINVAL
    assert call(o=S[0]) == EALIAS and call(o=S[1]) == EALIAS
    assert call(n=0) == OK
    need = L.embedding_grad_scratch_bytes(10, 7, 16)
    assert need > 0 and L.embedding_grad_scratch_bytes(0, 7, 16) == 0
    assert L.embedding_grad_scratch_bytes(10, 0, 16) == 0

    def grad(do=S[0], i=S[1], o=S[2], n=10, rows=7, d=16, st=16, ty=f32, it=i64, ot=f32, s=S[3], sb=need):
        return L.embedding_grad(do, i, o, n, rows, d, st, ty, it, ot, 1.0, s, sb, None)
    assert grad(ot=D["bf16"]) == ENOTSUP and grad(ty=D["bf16"], ot=D["f16"]) == ENOTSUP
    assert grad(do=None) == EINVAL and grad(o=None) == EINVAL and grad(s=None) == EINVAL
    assert grad(s=S[3] + 8) == EINVAL and grad(sb=need - 1) == ESCRATCH
    assert grad(o=S[0]) == EALIAS and grad(s=S[1]) == EALIAS and grad(s=S[2] + 16) == EALIAS
