"""What beam search refuses before anything is launched: sizes and views (no GPU needed)."""
import ctypes

import pytest
import torch

import stream_compaction_amd as sc
from stream_compaction_amd import beam
from test_sequence_refusals import OnGpu

EINVAL = 1


def test_rows_too_long_to_count():
    # in fewer than 2^47 bytes in all, but more workgroups than 32 bits count
    L, at = sc.lib(), ctypes.c_void_p * 1
    for size in (1 << 43, (1 << 46) + 3):
        for to in (1 << 12, 1 << 46):
            assert L.beam_reorder(at(1 << 12), at(to), (ctypes.c_int64 * 1)(size), 1, 1 << 47, 1, 1, None) == EINVAL, size


def test_conjugated_views(monkeypatch):
    # a view that torch conjugates only when it is read: its memory holds other values than it has
    reached = []
    monkeypatch.setattr(beam, "lib", lambda: type("L", (), {"beam_reorder": lambda self, *a: reached.append(1) or 0})())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    p = OnGpu(2, 3, dtype=torch.int32)
    plain, other = (OnGpu(2, 3, 5, dtype=torch.complex64) for _ in range(2))
    view = plain.conj()
    view.index = 0
    assert view.is_contiguous() and view.is_conj()
    for from_, to in (([view], [other]), ([plain], [other.conj()]), ([other, view], [plain, other])):
        for t in to:
            t.index = 0
        with pytest.raises(ValueError, match="conjugated"):
            beam.beam_reorder(from_, p, to)
    assert not reached
    beam.beam_reorder([view], p)                         # in place it stays what it is
    beam.beam_reorder([plain], p, [other])
    assert len(reached) == 2


def test_end_tokens(monkeypatch):
    reached = []

    class Library:
        def beam_select(self, args, *more):
            reached.append(args.end_token)
            return 0

        def beam_select_scratch_bytes(self, args):
            return 64
    monkeypatch.setattr(beam, "lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    x, s, done = OnGpu(2, 3, 50), OnGpu(2, 3), OnGpu(2, 3, dtype=torch.uint8)
    more = {"out_scores": OnGpu(2, 4), "parents": OnGpu(2, 4, dtype=torch.int32), "tokens": OnGpu(2, 4, dtype=torch.int32),
            "scratch": OnGpu(64, dtype=torch.uint8)}
    for wrong in (-1, 50, 1 << 64, (1 << 64) + 7, -(1 << 64) + 7):
        with pytest.raises(ValueError, match="end_token"):
            beam.beam_select(x, s, 4, finished=done, end_token=wrong, **more)
        beam.beam_select(x, s, 4, end_token=wrong, **more)   # not used without ended beams
    assert reached == [0] * 5
    beam.beam_select(x, s, 4, finished=done, end_token=49, **more)
    assert reached[-1] == 49
