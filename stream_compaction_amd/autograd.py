"""The sequence operators for torch's automatic differentiation.

``causal_conv``, ``selective_scan``, ``gated_scan`` and ``embedding`` take the arguments of the
functions of these names in ``stream_compaction_amd.sequence`` and can be differentiated with respect to
every floating input, through the output and the final state.  Both directions run in the
library's kernels on the current stream; work space comes from torch's allocator, so a
forward and backward pass can be captured into a HIP graph (of leaves that no output of
eager work still refers to: torch takes a leaf's gradient to the stream of the first graph that
holds it, and a capture that waits for another stream fails).  Gradients are taken once, in
reverse: there are no second derivatives, no forward mode and no ``torch.func`` transforms
(``grad``, ``vmap``, ...), which torch refuses with an error of its own.
"""
import torch

from . import sequence as _ops


def _rows(g, like):
    """A gradient with a contiguous last axis (a sum's is a single expanded element)."""
    if g is None:
        return torch.zeros(like.shape, dtype=like.dtype, device=like.device)
    return g if g.shape[-1] <= 1 or g.stride(-1) == 1 else g.contiguous()


def _dense(g):
    return None if g is None else g.contiguous()


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, lengths, silu):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, initial_state, lengths)
        ctx.silu = silu
        return _ops.causal_conv(x, weight, bias, initial_state, lengths, silu)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dfinal):
        x, weight, bias, initial_state, lengths = ctx.saved_tensors
        g = _ops.causal_conv_grad(_rows(dy, x), x, weight, bias, initial_state, lengths, ctx.silu,
                                  dfinal=_dense(dfinal))
        return g["dx"], g["dweight"], g["dbias"], g["dstate"], None, None


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, initial_state, lengths, softplus, recording):
        ctx.set_materialize_grads(False)
        more = {"D": D, "z": z, "dt_bias": dt_bias, "softplus": softplus, "lengths": lengths}
        # (an input that requires a gradient is said to need one under no_grad, too)
        if not (recording and any(ctx.needs_input_grad)):
            return _ops.selective_scan(x, dt, A, B, C, initial_state=initial_state, **more)
        y, state, starts = _ops.selective_scan(x, dt, A, B, C, initial_state=initial_state,
                                               keep_starts=True, **more)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, lengths, starts)
        ctx.softplus, ctx.has_state = softplus, initial_state is not None
        return y, state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dfinal):
        x, dt, A, B, C, D, z, dt_bias, lengths, starts = ctx.saved_tensors
        g = _ops.selective_scan_grad(_rows(dy, x), x, dt, A, B, C, starts, D=D, z=z,
                                     dt_bias=dt_bias, softplus=ctx.softplus, lengths=lengths,
                                     dfinal=_dense(dfinal))
        return (g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddt_bias"],
                g["dstate"] if ctx.has_state else None, None, None, None)


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, forget, rate, input_gate, z, initial_state, lengths, recording):
        ctx.set_materialize_grads(False)
        more = {"rate": rate, "input_gate": input_gate, "z": z, "lengths": lengths}
        # (an input that requires a gradient is said to need one under no_grad, too)
        if not (recording and any(ctx.needs_input_grad)):
            return _ops.gated_scan(x, forget, initial_state=initial_state, **more)
        y, state, starts = _ops.gated_scan(x, forget, initial_state=initial_state,
                                           keep_starts=True, **more)
        ctx.save_for_backward(x, forget, rate, input_gate, z, lengths, starts)
        ctx.has_state = initial_state is not None
        return y, state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dfinal):
        x, forget, rate, input_gate, z, lengths, starts = ctx.saved_tensors
        g = _ops.gated_scan_grad(_rows(dy, x), x, forget, starts, rate=rate,
                                 input_gate=input_gate, z=z, lengths=lengths,
                                 dfinal=_dense(dfinal))
        return (g["dx"], g["dforget"], g["drate"], g["dinput_gate"], g["dz"],
                g["dstate"] if ctx.has_state else None, None, None)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = weight.shape[0], scale
        return _ops.embedding(weight, ids, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        return _ops.embedding_grad(dout.contiguous(), ids, ctx.rows, ctx.scale), None, None


def causal_conv(x, weight, bias=None, initial_state=None, lengths=None, silu=True):
    """Differentiable ``sequence.causal_conv``: ``(y, final_state)``."""
    return _CausalConv.apply(x, weight, bias, initial_state, lengths, bool(silu))


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False,
                   initial_state=None, lengths=None):
    """Differentiable ``sequence.selective_scan``: ``(y, final_state)``."""
    return _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, initial_state, lengths,
                                bool(softplus), torch.is_grad_enabled())


def gated_scan(x, forget, rate=None, input_gate=None, z=None, initial_state=None, lengths=None):
    """Differentiable ``sequence.gated_scan``: ``(y, final_state)``."""
    return _GatedScan.apply(x, forget, rate, input_gate, z, initial_state, lengths,
                            torch.is_grad_enabled())


def embedding(weight, ids, scale=1.0):
    """Differentiable ``sequence.embedding``; the table's gradient has the table's type."""
    return _Embedding.apply(weight, ids, float(scale))
