"""Beam search over the library: the choice of the best continuations, and the beams' states
moved to where they go on.

Thin wrappers over the C ABI (``include/scan.h`` has every definition and rule), in the manner
of the sequence operators: they check shapes, types and devices, allocate what is not given, and
pass pointers and the current HIP stream, which must be of the data's GPU.
"""
from array import array

import torch

from . import check, lib
from ._sequence_abi import BeamArgs
from .sequence import _code, _like, _out, _queue, _require, _scratch


def beam_select(logits, scores, count, finished=None, end_token=0, out_scores=None, parents=None,
                tokens=None, scratch=None, stream=None):
    """The ``count`` best continuations (1 to 64) of each batch entry over its beams (1 to 64) and
    the vocabulary.

    ``logits`` is ``[batch, beams, vocab]`` float32, float16 or bfloat16, contiguous along the
    vocabulary, and ``scores`` (float32 ``[batch, beams]``) the beams' own.  A continuation's score
    is its beam's plus the token's log softmax, formed in 64 bits.  ``finished`` (uint8 or bool
    ``[batch, beams]``) marks beams that have ended: such a beam goes on by ``end_token`` alone, at
    its own score.  Logits of -infinity (or NaN) are masked.

    Returns ``(out_scores, parents, tokens)``, each ``[batch, count]`` (float32, int32, int32), the
    best first; of equal scores the lower beam, then the greater logit, then the lower token.
    """
    _require(logits.dim() == 3, "logits must be [batch, beams, vocab]")
    _require(logits.is_cuda, "logits must be a GPU tensor")
    code, dev = _code(logits, "logits"), logits.get_device()
    b, k, v = logits.shape
    stride = logits.stride()
    _require(v <= 1 or stride[2] == 1, "logits must have a contiguous last axis")
    count = int(count)
    _require(count >= 1, "count must be at least 1")
    sp = _like(scores, "scores", (b, k), torch.float32, dev)
    fp = None
    if finished is not None:
        if finished.dtype is torch.bool:
            finished = finished.view(torch.uint8)
        fp = _like(finished, "finished", (b, k), torch.uint8, dev)
        end_token = int(end_token)
        # (here, as a number beyond 64 bits would reach the library as another)
        _require(0 <= end_token < v, "end_token must be in the vocabulary")
    else:
        end_token = 0
    a = BeamArgs(logits.data_ptr(), sp, fp, b, k, v, count, end_token, stride[0], stride[1], code)
    chosen = (b, count)
    out_scores = _out(out_scores, "out_scores", chosen, torch.float32, scores, stream)
    parents = _out(parents, "parents", chosen, torch.int32, out_scores, stream)
    tokens = _out(tokens, "tokens", chosen, torch.int32, parents, stream)
    L = lib()
    scratch, room = _scratch(scratch, L.beam_select_scratch_bytes(a), scores, stream)
    check(L.beam_select(a, out_scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                        scratch.data_ptr(), room, _queue(stream, dev)))
    return out_scores, parents, tokens


def _pointers(tensors, what, dev):
    for t in tensors:
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous tensors on cuda:{dev}")
    return array("Q", [t.data_ptr() for t in tensors])


def beam_reorder(states, parents, new_states=None, stream=None):
    """The beams' states follow them: ``new[b, j] = old[b, parents[b, j]]`` in each of ``states``,
    a list of contiguous tensors of any type, ``[batch, beams, ...]`` or ``[batch * beams, ...]``
    (at most 1024, moved together).

    ``parents`` is int32 ``[batch, beams]`` (1 to 64 beams); an entry outside ``[0, beams)`` counts
    as the beam's own.  The states are moved in place, where beams that go on as themselves are
    neither read nor written, or into ``new_states``, tensors of the same shapes and types that
    overlap nothing.  Returns the list of the moved tensors.
    """
    _require(parents.dim() == 2 and parents.is_cuda, "parents must be a GPU tensor [batch, beams]")
    dev = parents.get_device()
    b, k = parents.shape
    pp = _like(parents, "parents", (b, k), torch.int32, dev)
    states = list(states)
    out = states if new_states is None else list(new_states)
    _require(len(out) == len(states), "new_states must have as many tensors as states")
    n = len(states)
    _require(n <= 1024, "at most 1024 states")
    # (up to a thousand tensors a token: each is asked little, and the pointers go out in arrays)
    rows, shapes = b * k, [t.shape for t in states]
    for shape in set(shapes):
        if not (len(shape) > 0 and (shape[0] == rows or shape[:2] == (b, k))):
            raise ValueError("states must be [batch, beams, ...] or [batch * beams, ...]")
    from_ = to = _pointers(states, "states", dev)
    if new_states is not None:
        types = [t.dtype for t in states]
        if [t.shape for t in out] != shapes or [t.dtype for t in out] != types:
            raise ValueError("new_states must have the shapes and types of states")
        # (what is moved is memory, which holds the conjugate of a lazily conjugated view's values)
        if any(ty.is_complex for ty in set(types)) and [t.is_conj() for t in out] != [t.is_conj() for t in states]:
            raise ValueError("new_states must be conjugated views exactly where states are")
        to = _pointers(out, "new_states", dev)
    sizes = array("q", [t.nbytes // rows for t in states] if rows else [0] * n)
    check(lib().beam_reorder(from_.buffer_info()[0], to.buffer_info()[0], sizes.buffer_info()[0], n, pp, b, k,
                             _queue(stream, dev)))
    return out
