"""The oracle of beam search against choices made by hand, and what its entry points refuse (needs
no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import beam_ref as ref
import stream_compaction_amd as sc
from stream_compaction_amd import beam
from stream_compaction_amd._sequence_abi import BeamArgs
from test_sequence_refusals import OnGpu

OK, EINVAL, ENOTSUP, EALIAS, ESCRATCH = range(5)
S = [0x10000000 * (i + 1) for i in range(24)]
INF = float("inf")


def test_by_hand():
    logits = np.log(np.array([[[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]]))
    scores = np.log(np.array([[0.5, 0.5]]))
    s, p, t = ref.select(logits, scores, 6)
    assert np.allclose(np.exp(s[0]), [0.4, 0.25, 0.125, 0.125, 0.05, 0.05])
    assert p[0].tolist() == [1, 0, 0, 0, 1, 1] and t[0].tolist() == [1, 0, 1, 2, 0, 2]
    # a finished beam goes on by the end token alone
    s, p, t = ref.select(logits, scores, 6, np.array([[1, 0]]), 2)
    assert p[0].tolist() == [0, 1, 1, 1, 0, 0] and t[0].tolist() == [2, 1, 0, 2, 0, 1]
    assert s[0, 0] == scores[0, 0] and s[0, 4] == -INF


def test_masked_and_infinite():
    logits = np.array([[[-INF, -INF], [INF, 3.0], [np.nan, 1.0]]])
    s, p, t = ref.select(logits, np.zeros((1, 3)), 6)
    assert p[0].tolist() == [1, 2, 0, 0, 1, 2] and t[0].tolist() == [0, 1, 0, 1, 1, 0]
    assert s[0, :2].tolist() == [0.0, 0.0] and (s[0, 2:] == -INF).all()


@pytest.fixture
def library(monkeypatch):
    class Refuses:
        def __getattr__(self, name):
            def no_library(*args):
                raise AssertionError("a refused call reached the library")
            return (lambda *a: 64) if name.endswith("_bytes") else no_library
    monkeypatch.setattr(beam, "lib", Refuses)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)


def outs():
    i = torch.int32
    return {"out_scores": OnGpu(2, 4), "parents": OnGpu(2, 4, dtype=i), "tokens": OnGpu(2, 4, dtype=i),
            "scratch": OnGpu(64, dtype=torch.uint8)}


@pytest.mark.usefixtures("library")
def test_refused_by_the_python_side():
    x, s = OnGpu(2, 3, 50), OnGpu(2, 3)
    with pytest.raises(AssertionError, match="reached"):
        beam.beam_select(x, s, 4, **outs())
    for wrong in (dict(logits=OnGpu(6, 50)), dict(logits=torch.zeros(2, 3, 50)), dict(logits=OnGpu(2, 3, 100)[..., ::2]),
                  dict(scores=OnGpu(2, 4)), dict(scores=OnGpu(2, 3, dtype=torch.float64)), dict(scores=OnGpu(2, 3, index=1)),
                  dict(count=0), dict(count=5), dict(finished=OnGpu(2, 3)), dict(finished=OnGpu(3, 3, dtype=torch.uint8)),
                  dict(parents=OnGpu(2, 4, dtype=torch.int64)), dict(scratch=OnGpu(64))):
        k = {"logits": x, "scores": s, "count": 4, **outs(), **wrong}
        with pytest.raises(ValueError):
            beam.beam_select(**k)
    for ty in (torch.float64, torch.int32):
        with pytest.raises(NotImplementedError):
            beam.beam_select(OnGpu(2, 3, 50, dtype=ty), s, 4)
    p = OnGpu(2, 3, dtype=torch.int32)
    good = [OnGpu(2, 3, 7), OnGpu(6, 5, dtype=torch.bfloat16), OnGpu(6)]
    with pytest.raises(AssertionError, match="reached"):
        beam.beam_reorder(good, p)
    with pytest.raises(AssertionError, match="reached"):
        beam.beam_reorder(good, p, [t.clone() for t in good])
    for wrong in ([OnGpu(3, 2, 7)], [OnGpu(2, 7)], [OnGpu()], [OnGpu(2, 3, 8)[..., ::2]], [OnGpu(2, 3, 7, index=1)],
                  [OnGpu(2, 3)] * 1025):
        with pytest.raises(ValueError):
            beam.beam_reorder(wrong, p)
    for wrong in ([OnGpu(2, 3, 7)], [OnGpu(2, 3, 8), good[1], good[2]], [good[0].half(), good[1], good[2]]):
        with pytest.raises(ValueError):
            beam.beam_reorder(good, p, wrong)
    for wrong in (OnGpu(6, dtype=torch.int32), OnGpu(2, 3), OnGpu(2, 3, dtype=torch.int64), torch.zeros(2, 3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            beam.beam_reorder(good, wrong)


@pytest.mark.usefixtures("library")
def test_data_of_another_gpu_than_the_stream(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        beam.beam_select(OnGpu(2, 3, 50), OnGpu(2, 3), 4, **outs())
    with pytest.raises(ValueError, match="cuda:1"):
        beam.beam_reorder([OnGpu(2, 3, 7)], OnGpu(2, 3, dtype=torch.int32))


def args(**more):
    k = dict(logits=S[0], scores=S[1], batch=2, beams=3, vocab=100, count=6, logits_batch=300, logits_beam=100,
             dtype=sc.DTYPE_CODES["f32"])
    k.update(more)
    return BeamArgs(**k)


def test_refused_selections():
    L, room = sc.lib(), 1 << 46
    call = lambda a, o=S[3], p=S[4], t=S[5], s=S[6], n=room: L.beam_select(a, o, p, t, s, n, None)  # noqa: E731
    assert call(args(batch=0), None, None, None, None, 0) == OK
    for wrong in (dict(batch=-1), dict(batch=1 << 31), dict(beams=0), dict(vocab=0), dict(vocab=1 << 31), dict(count=0),
                  dict(count=7, beams=1, vocab=6), dict(logits=None), dict(scores=None), dict(logits=S[0] + 2),
                  dict(logits_batch=-300), dict(finished=S[2], end_token=100), dict(finished=S[2], end_token=-1),
                  dict(batch=1 << 30, logits_batch=1 << 30, logits_beam=1),
                  dict(batch=(1 << 31) - 1, beams=64, vocab=(1 << 31) - 1, logits_batch=0, logits_beam=0)):
        assert call(args(**wrong)) == EINVAL, wrong
    assert L.beam_select_scratch_bytes(args(batch=(1 << 31) - 1, beams=64, vocab=(1 << 31) - 1)) == 0
    for wrong in (dict(beams=65), dict(count=65), dict(dtype=sc.DTYPE_CODES["f64"])):
        assert call(args(**wrong)) == ENOTSUP, wrong
        assert L.beam_select_scratch_bytes(args(**wrong)) == 0
    assert call(None) == EINVAL
    need = L.beam_select_scratch_bytes(args())
    assert need > 0 and call(args(), n=need - 1) == ESCRATCH
    assert call(args(), s=S[6] + 8) == EINVAL and call(args(), s=None) == EINVAL
    assert call(args(), o=None) == EINVAL and call(args(), t=None) == EINVAL
    for wrong in (dict(o=S[0]), dict(p=S[1]), dict(t=S[4] + 4), dict(s=S[0] + 2384)):
        assert call(args(), **wrong) == EALIAS, wrong
    assert call(args(finished=S[3])) == EALIAS


def test_refused_reorders():
    L = sc.lib()

    def call(from_, to, size, batch=2, beams=3, parents=S[20], n=None):
        n = len(from_) if n is None else n
        return L.beam_reorder((ctypes.c_void_p * max(n, 1))(*from_), (ctypes.c_void_p * max(n, 1))(*to),
                              (ctypes.c_int64 * max(n, 1))(*size), n, parents, batch, beams, None)
    assert call([], [], []) == OK and call([None], [None], [0], batch=0) == OK
    assert call([S[0]], [S[1]], [8], batch=-1) == EINVAL and call([S[0]], [S[1]], [8], batch=1 << 31) == EINVAL
    assert call([S[0]], [S[1]], [8], beams=0) == EINVAL and call([S[0]], [S[1]], [8], beams=65) == ENOTSUP
    assert call([S[0]], [S[1]], [-8]) == EINVAL and call([S[0]], [None], [8]) == EINVAL
    assert call([None], [S[1]], [8]) == EINVAL and call([S[0]], [S[1]], [1 << 45]) == EINVAL
    assert call([S[0]], [S[1]], [8], parents=None) == EINVAL and call([S[0]], [S[1]], [8], parents=S[20] + 2) == EINVAL
    assert L.beam_reorder(None, None, None, 1, S[20], 2, 3, None) == EINVAL
    assert L.beam_reorder(None, None, None, 1025, S[20], 2, 3, None) == EINVAL
    # 6 rows of 8 bytes: 48 bytes each
    for from_, to in (([S[0]], [S[0] + 8]), ([S[0]], [S[0] - 40]), ([S[0], S[0]], [S[0], S[0]]), ([S[0], S[1]], [S[1], S[2]]),
                      ([S[0], S[1]], [S[2], S[2] + 47]), ([S[0]], [S[20]]), ([S[20] + 20], [S[20] + 20]),
                      ([S[0], S[1]], [S[2], S[0] + 16])):
        assert call(from_, to, [8] * len(from_)) == EALIAS, (from_, to)


def test_struct_size():
    assert ctypes.sizeof(BeamArgs) == 88
