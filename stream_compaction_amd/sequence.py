"""Sequence operators of the library: causal convolution, selective scan, gated scan and token
embedding, each with its gradient, and the first three with their single-token step.

Thin wrappers over the C ABI (``include/scan.h`` has every definition and rule): they
check shapes, types and devices, allocate what is not given, and pass pointers, strides and
the current HIP stream, which must be of the data's GPU (as must a ``stream`` that is
given).  Activations are ``[batch, length, channels]`` float32, float16 or bfloat16 tensors
with contiguous channels; parameters and the scans' states are float32.
``stream_compaction_amd.autograd`` has the same operators for torch's automatic
differentiation.
"""
import ctypes

import torch

from . import DTYPE_CODES, check, lib
from ._sequence_abi import ConvArgs, GatedArgs, GatedGrads, ScanArgs, ScanGrads

_ACT = {torch.float32: DTYPE_CODES["f32"], torch.float16: DTYPE_CODES["f16"],
        torch.bfloat16: DTYPE_CODES["bf16"]}
_IDS = {torch.int32: DTYPE_CODES["i32"], torch.int64: DTYPE_CODES["i64"]}

_i64 = ctypes.c_int64


def _require(ok, message):
    if not ok:
        raise ValueError(message)


def _code(x, what):
    if x.dtype not in _ACT:
        raise NotImplementedError(f"{what}: dtype {x.dtype} is not supported")
    return _ACT[x.dtype]


# Devices are compared by index and new tensors made like existing ones where that serves:
# a step for one token is bound by this side, and both cost half of the plain way.
def _like(t, what, shape, dtype, dev):
    """Pointer of a contiguous tensor of this shape, type and GPU."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"cuda:{dev}")
    return t.data_ptr()


def _opt(t, what, shape, dtype, dev):
    return None if t is None else _like(t, what, shape, dtype, dev)


def _rows(t, what, shape, dtype, dev):
    """An activation tensor: shape, type, GPU, contiguous last axis."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have a contiguous last axis")
    return t.data_ptr()


def _queue(stream, dev):
    """The stream a call goes to, as a raw handle: one of the data's GPU, which a kernel of
    another GPU could not read."""
    if stream is not None:
        at = stream.device_index
    else:
        at = torch._C._cuda_getDevice()
    if at != dev:
        raise ValueError(f"the data is on cuda:{dev}, the stream on cuda:{at}")
    # (the raw handle: a Stream object costs more than the rest of a small call)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _new(shape, dtype, like, stream):
    """A new tensor on ``like``'s GPU.  Memory for an explicit stream comes from that stream's
    pool, so that it is not handed on while the stream still works on it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=like.device)
    if like.shape == shape and like.is_contiguous():
        return torch.empty_like(like) if like.dtype is dtype else torch.empty_like(like, dtype=dtype)
    if like.dtype is dtype:
        return like.new_empty(shape)
    return torch.empty(shape, dtype=dtype, device=like.device)


def _out(t, what, shape, dtype, like, stream):
    if t is None:
        return _new(shape, dtype, like, stream)
    _like(t, what, shape, dtype, like.get_device())
    return t


def _scratch(scratch, need, like, stream):
    """Scratch memory and its bytes; a float32 ``like`` makes it the cheapest."""
    if scratch is None:
        return _new((max(need, 16) + 3) // 4, torch.float32, like, stream), need
    if scratch.dtype != torch.uint8 or scratch.get_device() != like.get_device() or \
            not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous uint8 tensor on the data's device")
    return scratch, scratch.numel()


def _conv_args(x, weight, bias, initial_state, lengths, silu, step):
    if x.dim() != (2 if step else 3):
        raise ValueError("x must be [batch, channels]" if step else
                         "x must be [batch, length, channels]")
    _require(x.is_cuda, "x must be a GPU tensor")
    code = _code(x, "x")
    shape, dev, stride = x.shape, x.get_device(), x.stride()
    b, d = shape[0], shape[-1]
    _require(weight.dim() == 2, "weight must be [channels, width]")
    w = weight.shape[1]
    return ConvArgs(
        _rows(x, "x", shape, x.dtype, dev),
        _like(weight, "weight", (d, w), torch.float32, dev),
        _opt(bias, "bias", (d,), torch.float32, dev),
        _opt(initial_state, "initial_state", (b, w - 1, d), x.dtype, dev),
        _opt(lengths, "lengths", (b,), torch.int32, dev),
        b, 1 if step else shape[1], d, w,
        (stride[0], 0 if step else stride[1]), 1 if silu else 0, code)


def causal_conv(x, weight, bias=None, initial_state=None, lengths=None, silu=True, out=None,
                final_state=None, stream=None):
    """Causal convolution of ``x`` along time, one filter ``weight[channel]`` (float32
    ``[channels, width]``, width 1 to 8) per channel, then ``silu`` when asked.

    ``initial_state`` (``[batch, width - 1, channels]``) holds the inputs before the first
    token; ``lengths`` (int32 ``[batch]``) the tokens of each sequence that exist.  Returns
    ``(y, final_state)``: the second is the next call's initial state.
    """
    a = _conv_args(x, weight, bias, initial_state, lengths, silu, False)
    y = _out(out, "out", x.shape, x.dtype, x, stream)
    fs = _out(final_state, "final_state", (a.batch, a.width - 1, a.channels), x.dtype, x, stream)
    check(lib().causal_conv(a, y.data_ptr(), fs.data_ptr(), _queue(stream, x.get_device())))
    return y, fs


def causal_conv_grad(dy, x, weight, bias=None, initial_state=None, lengths=None, silu=True,
                     dfinal=None, scratch=None, stream=None):
    """Gradients of ``causal_conv`` from ``dy`` (and ``dfinal``, of the final state): a dict
    with ``dx``, ``dweight``, ``dbias`` and ``dstate`` (of the initial state; both None when
    that input is)."""
    a = _conv_args(x, weight, bias, initial_state, lengths, silu, False)
    dev, state = x.get_device(), (a.batch, a.width - 1, a.channels)
    dyp = _rows(dy, "dy", x.shape, x.dtype, dev)
    df = _opt(dfinal, "dfinal", state, x.dtype, dev)
    dx = _new(x.shape, x.dtype, x, stream)
    dw = _new(weight.shape, torch.float32, weight, stream)
    db = None if bias is None else _new(bias.shape, torch.float32, bias, stream)
    ds = None if initial_state is None else _new(state, x.dtype, initial_state, stream)
    L = lib()
    scratch, room = _scratch(scratch, L.causal_conv_grad_scratch_bytes(a), weight, stream)
    check(L.causal_conv_grad(a, dyp, (_i64 * 2)(*dy.stride()[:2]), df, dx.data_ptr(),
                             dw.data_ptr(), None if db is None else db.data_ptr(),
                             None if ds is None else ds.data_ptr(), scratch.data_ptr(),
                             room, _queue(stream, dev)))
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}


def causal_conv_step(state, x, weight, bias=None, silu=True, new_state=None, out=None,
                     stream=None):
    """One token of ``causal_conv``: ``x`` is ``[batch, channels]`` and ``state`` the last
    ``width - 1`` inputs, replaced by those that include ``x`` (in place, or into
    ``new_state``).  ``batch * channels`` is at most 2^31 - 1.  Returns ``y``."""
    a = _conv_args(x, weight, bias, None, None, silu, True)
    shape = (a.batch, a.width - 1, a.channels)
    dev = x.get_device()
    sp = _like(state, "state", shape, x.dtype, dev)
    np_ = sp if new_state is None else _like(new_state, "new_state", shape, x.dtype, dev)
    y = _out(out, "out", x.shape, x.dtype, x, stream)
    check(lib().causal_conv_step(a, sp, np_, y.data_ptr(), _queue(stream, dev)))
    return y


def _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, lengths, step):
    if x.dim() != (2 if step else 3):
        raise ValueError("x must be [batch, channels]" if step else
                         "x must be [batch, length, channels]")
    _require(x.is_cuda, "x must be a GPU tensor")
    code = _code(x, "x")
    dev, ty = x.get_device(), x.dtype
    shape = x.shape
    b, d = shape[0], shape[-1]
    _require(A.dim() == 2, "A must be [channels, states]")
    n = A.shape[1]
    _require(B.dim() == x.dim() + 1, "B must be [batch, length, groups, states] (a step: "
                                     "[batch, groups, states])")
    groups = B.shape[-2]
    rows = shape[:-1] + (groups, n)
    # (shapes before strides: an argument of another rank has not as many)
    xp, dtp = _rows(x, "x", shape, ty, dev), _rows(dt, "dt", shape, ty, dev)
    Bp, Cp = _rows(B, "B", rows, ty, dev), _rows(C, "C", rows, ty, dev)
    zp = None if z is None else _rows(z, "z", shape, ty, dev)
    length, zs = 1, (0, 0)
    if step:
        xs, ds = (x.stride(0), 0), (dt.stride(0), 0)
        Bs, Cs = (B.stride(0), 0, B.stride(1)), (C.stride(0), 0, C.stride(1))
        if z is not None:
            zs = (z.stride(0), 0)
    else:
        length = shape[1]
        xs, ds, Bs, Cs = x.stride()[:2], dt.stride()[:2], B.stride()[:3], C.stride()[:3]
        if z is not None:
            zs = z.stride()[:2]
    f32 = torch.float32
    return ScanArgs(
        xp, dtp, Bp, Cp, zp,
        _like(A, "A", (d, n), f32, dev), None if D is None else _like(D, "D", (d,), f32, dev),
        None if dt_bias is None else _like(dt_bias, "dt_bias", (d,), f32, dev),
        None if initial_state is None else
        _like(initial_state, "initial_state", (b, d, n), f32, dev),
        None if lengths is None else _like(lengths, "lengths", (b,), torch.int32, dev),
        b, length, d, n, groups, xs, ds, zs, Bs, Cs, 1 if softplus else 0, code)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False,
                   initial_state=None, lengths=None, keep_starts=False, out=None,
                   final_state=None, stream=None):
    """Selective state space scan.

    ``x``, ``dt`` and the gate ``z`` are ``[batch, length, channels]``, ``B`` and ``C``
    ``[batch, length, groups, states]`` (channel ``c`` uses group ``c // (channels //
    groups)``), ``A`` float32 ``[channels, states]`` (1 to 64 states), ``D`` and ``dt_bias``
    float32 ``[channels]``.  Per channel, ``s = dt + dt_bias`` (through softplus when asked),
    ``h = exp(s A) h + s x B`` and ``y = (C . h + D x) silu(z)``.

    Returns ``(y, final_state)``, the state float32 ``[batch, channels, states]``; with
    ``keep_starts`` also what ``selective_scan_grad`` needs of this call.
    """
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, lengths, False)
    y = _out(out, "out", x.shape, x.dtype, x, stream)
    fs = _out(final_state, "final_state", (a.batch, a.channels, a.states), torch.float32,
              A if initial_state is None else initial_state, stream)
    L = lib()
    starts = None
    if keep_starts:
        starts = _new((L.selective_scan_starts_bytes(a) // 4,), torch.float32, A, stream)
    sp = None if starts is None else starts.data_ptr()
    # (short scans are never split)
    need = L.selective_scan_split_scratch_bytes(a) if x.shape[1] >= 512 else 0
    if need == 0:
        check(L.selective_scan(a, y.data_ptr(), fs.data_ptr(), sp, _queue(stream, x.get_device())))
    else:
        scratch, room = _scratch(None, need, A, stream)
        check(L.selective_scan_split(a, y.data_ptr(), fs.data_ptr(), sp, scratch.data_ptr(), room,
                                     _queue(stream, x.get_device())))
    return (y, fs, starts) if keep_starts else (y, fs)


def selective_scan_grad(dy, x, dt, A, B, C, starts, D=None, z=None, dt_bias=None, softplus=False,
                        lengths=None, dfinal=None, scratch=None, stream=None):
    """Gradients of ``selective_scan`` called with the same arguments and ``keep_starts``,
    from ``dy`` (and ``dfinal``, of the final state): a dict with ``dx``, ``ddt``, ``dA``,
    ``dB``, ``dC``, ``dD``, ``dz``, ``ddt_bias`` (None where that input is) and ``dstate``
    (of the initial state)."""
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, None, lengths, False)
    dev, ty, f32 = x.get_device(), x.dtype, torch.float32
    state = (a.batch, a.channels, a.states)
    L = lib()
    dyp = _rows(dy, "dy", x.shape, ty, dev)
    df = _opt(dfinal, "dfinal", state, f32, dev)
    sp = _like(starts, "starts", (L.selective_scan_starts_bytes(a) // 4,), f32, dev)
    out = {"dx": _new(x.shape, ty, x, stream), "ddt": _new(x.shape, ty, x, stream),
           "dA": _new(A.shape, f32, A, stream), "dB": _new(B.shape, ty, B, stream),
           "dC": _new(B.shape, ty, B, stream),
           "dD": None if D is None else _new(D.shape, f32, D, stream),
           "dz": None if z is None else _new(x.shape, ty, x, stream),
           "ddt_bias": None if dt_bias is None else _new(dt_bias.shape, f32, dt_bias, stream),
           "dstate": _new(state, f32, A, stream)}
    p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
    g = ScanGrads(dyp, dy.stride()[:2], df, sp, p["dx"], p["ddt"], p["dB"], p["dC"], p["dz"],
                  p["dA"], p["dD"], p["ddt_bias"], p["dstate"])
    scratch, room = _scratch(scratch, L.selective_scan_grad_scratch_bytes(a), A, stream)
    check(L.selective_scan_grad(a, g, scratch.data_ptr(), room, _queue(stream, dev)))
    return out


def selective_scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False,
                        new_state=None, out=None, stream=None):
    """One token of ``selective_scan``: ``x``, ``dt``, ``z`` are ``[batch, channels]``, ``B``
    and ``C`` ``[batch, groups, states]``; ``state`` (float32 ``[batch, channels, states]``)
    moves on in place, or into ``new_state``.  ``batch * channels`` is at most 2^27 - 1.
    Returns ``y``."""
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, None, None, True)
    shape = (a.batch, a.channels, a.states)
    dev = x.get_device()
    sp = _like(state, "state", shape, torch.float32, dev)
    np_ = sp if new_state is None else _like(new_state, "new_state", shape, torch.float32, dev)
    y = _out(out, "out", x.shape, x.dtype, x, stream)
    check(lib().selective_scan_step(a, sp, np_, y.data_ptr(), _queue(stream, dev)))
    return y


def _gated_args(x, forget, rate, input_gate, z, initial_state, lengths, step):
    shape = x.shape
    if len(shape) != (2 if step else 3):
        raise ValueError("x must be [batch, channels]" if step else
                         "x must be [batch, length, channels]")
    _require(x.is_cuda, "x must be a GPU tensor")
    code = _code(x, "x")
    dev, ty, f32 = x.get_device(), x.dtype, torch.float32
    b, d = shape[0], shape[-1]
    # (shapes before strides: an argument of another rank has not as many)
    xp, fp = _rows(x, "x", shape, ty, dev), _rows(forget, "forget", shape, ty, dev)
    xs, fs, gs, zs = x.stride(), forget.stride(), (0, 0), (0, 0)
    ip = zp = None
    if input_gate is not None:
        ip, gs = _rows(input_gate, "input_gate", shape, ty, dev), input_gate.stride()
    if z is not None:
        zp, zs = _rows(z, "z", shape, ty, dev), z.stride()
    # (a step has no token axis; what stands in its place is not used)
    return GatedArgs(
        xp, fp, ip, zp, None if rate is None else _like(rate, "rate", (d,), f32, dev),
        None if initial_state is None else
        _like(initial_state, "initial_state", (b, d), f32, dev),
        None if lengths is None else _like(lengths, "lengths", (b,), torch.int32, dev),
        b, 1 if step else shape[1], d, xs[0], xs[1], fs[0], fs[1], gs[0], gs[1], zs[0], zs[1], code)


def gated_scan(x, forget, rate=None, input_gate=None, z=None, initial_state=None, lengths=None,
               keep_starts=False, out=None, final_state=None, scratch=None, stream=None):
    """Gated scan: one state per channel, moved by gates that depend on the token.

    ``x``, ``forget`` and, when given, ``input_gate`` and the output gate ``z`` are ``[batch,
    length, channels]``.  With ``s = sigmoid(forget)`` and ``v = sigmoid(input_gate)`` (1
    without one), the state moves by ``h = a h + w v x`` and ``y = h silu(z)``, where

    * without ``rate``: ``a = s`` and ``w = 1 - s``, a convex average;
    * with ``rate`` (float32 ``[channels]``, 0 or greater): ``a = exp(-rate s)`` and ``w =
      sqrt(1 - a^2)``, which keeps the state's variance at the input's.

    Returns ``(y, final_state)``, the state float32 ``[batch, channels]``; with
    ``keep_starts`` also what ``gated_scan_grad`` needs of this call.
    """
    a = _gated_args(x, forget, rate, input_gate, z, initial_state, lengths, False)
    y = _out(out, "out", x.shape, x.dtype, x, stream)
    f32 = torch.float32
    fs = _out(final_state, "final_state", (a.batch, a.channels), f32, x if rate is None else rate, stream)
    L = lib()
    starts = None
    if keep_starts:
        starts = _new((L.gated_scan_starts_bytes(a) // 4,), f32, fs, stream)
    sp = None if starts is None else starts.data_ptr()
    need = L.gated_scan_scratch_bytes(a)
    scratch_p, room = None, 0
    if need or scratch is not None:
        scratch, room = _scratch(scratch, need, fs, stream)
        scratch_p = scratch.data_ptr()
    check(L.gated_scan(a, y.data_ptr(), fs.data_ptr(), sp, scratch_p, room,
                       _queue(stream, x.get_device())))
    return (y, fs, starts) if keep_starts else (y, fs)


def gated_scan_grad(dy, x, forget, starts, rate=None, input_gate=None, z=None, lengths=None,
                    dfinal=None, scratch=None, stream=None):
    """Gradients of ``gated_scan`` called with the same arguments and ``keep_starts``, from
    ``dy`` (and ``dfinal``, of the final state): a dict with ``dx``, ``dforget``, ``drate``,
    ``dinput_gate``, ``dz`` (None where that input is) and ``dstate`` (of the initial state).
    A rate of 0 or below, where the weight has no derivative, gets a gradient of 0."""
    a = _gated_args(x, forget, rate, input_gate, z, None, lengths, False)
    dev, ty, f32 = x.get_device(), x.dtype, torch.float32
    L = lib()
    dyp = _rows(dy, "dy", x.shape, ty, dev)
    df = _opt(dfinal, "dfinal", (a.batch, a.channels), f32, dev)
    sp = _like(starts, "starts", (L.gated_scan_starts_bytes(a) // 4,), f32, dev)
    out = {"dx": _new(x.shape, ty, x, stream), "dforget": _new(x.shape, ty, x, stream),
           "drate": None if rate is None else _new(rate.shape, f32, rate, stream),
           "dinput_gate": None if input_gate is None else _new(x.shape, ty, x, stream),
           "dz": None if z is None else _new(x.shape, ty, x, stream),
           "dstate": _new((a.batch, a.channels), f32, starts, stream)}
    p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
    g = GatedGrads(dyp, dy.stride()[:2], df, sp, p["dx"], p["dforget"], p["dinput_gate"], p["dz"],
                   p["drate"], p["dstate"])
    scratch, room = _scratch(scratch, L.gated_scan_grad_scratch_bytes(a), starts, stream)
    check(L.gated_scan_grad(a, g, scratch.data_ptr(), room, _queue(stream, dev)))
    return out


def gated_scan_step(state, x, forget, rate=None, input_gate=None, z=None, new_state=None, out=None,
                    stream=None):
    """One token of ``gated_scan``: ``x``, ``forget``, ``input_gate`` and ``z`` are ``[batch,
    channels]``; ``state`` (float32 ``[batch, channels]``) moves on in place, or into
    ``new_state``.  ``batch * channels`` is at most 2^31 - 1.  Returns ``y``."""
    a = _gated_args(x, forget, rate, input_gate, z, None, None, True)
    shape = (a.batch, a.channels)
    dev = x.get_device()
    sp = _like(state, "state", shape, torch.float32, dev)
    np_ = sp if new_state is None else _like(new_state, "new_state", shape, torch.float32, dev)
    y = _out(out, "out", x.shape, x.dtype, x, stream)
    check(lib().gated_scan_step(a, sp, np_, y.data_ptr(), _queue(stream, dev)))
    return y


def _table(t, what):
    """A [rows, channels] tensor with contiguous channels: its type code and row stride."""
    _require(t.dim() == 2 and t.is_cuda, f"{what} must be a 2-D GPU tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return _code(t, what), t.stride(0)


def _id_code(ids, dev):
    if ids.dtype not in _IDS:
        raise NotImplementedError(f"ids: dtype {ids.dtype} is not supported")
    if ids.get_device() != dev or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous tensor on cuda:{dev}")
    return _IDS[ids.dtype]


def embedding(weight, ids, scale=1.0, out=None, stream=None):
    """``scale * weight[ids]`` for int32 or int64 ``ids`` of any shape; ids outside the table
    are masked tokens and give zeros.  Returns ``[*ids.shape, channels]`` in weight's type."""
    code, stride = _table(weight, "weight")
    idc = _id_code(ids, weight.get_device())
    rows, d = weight.shape
    out = _out(out, "out", ids.shape + (d,), weight.dtype, weight, stream)
    check(lib().embedding(weight.data_ptr(), ids.data_ptr(), out.data_ptr(), ids.numel(), rows, d,
                          stride, code, idc, float(scale), _queue(stream, weight.get_device())))
    return out


def embedding_grad(dout, ids, rows, scale=1.0, dtype=None, out=None, scratch=None, stream=None):
    """Gradient of ``embedding``'s table: ``[rows, channels]`` in ``dtype`` (dout's, or
    float32), row ``v`` being ``scale`` times the sum of ``dout`` over the tokens with id
    ``v``; masked tokens add nothing.  The same bits every time."""
    if dout.dim() == 0 or dout.shape[:-1] != ids.shape:
        raise ValueError("dout must be [*ids.shape, channels]")
    d = dout.shape[-1]
    flat = dout
    if dout.dim() != 2:
        try:
            flat = dout.view(ids.numel(), d)
        except RuntimeError:
            raise ValueError("dout's rows must lie at one stride") from None
    code, stride = _table(flat, "dout")
    idc = _id_code(ids, dout.get_device())
    dtype = dtype or (out.dtype if out is not None else dout.dtype)
    if dtype not in (dout.dtype, torch.float32):
        raise NotImplementedError("the gradient is of dout's type or float32")
    out = _out(out, "out", (int(rows), d), dtype, dout, stream)
    L = lib()
    n = ids.numel()
    scratch, room = _scratch(scratch, L.embedding_grad_scratch_bytes(n, rows, d), dout, stream)
    check(L.embedding_grad(flat.data_ptr(), ids.data_ptr(), out.data_ptr(), n, rows, d, stride,
                           code, idc, _ACT[dtype], float(scale), scratch.data_ptr(),
                           room, _queue(stream, dout.get_device())))
    return out
