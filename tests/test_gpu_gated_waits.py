"""Waits of the gated scan that end without what they wait for: in a build that asks once for a word and never writes
some, forward and gradient end, what depends on a lost word is no number, and everything else is right or no number."""
import pytest
import torch

import stream_compaction_amd as sc
from stream_compaction_amd import build
from stream_compaction_amd._sequence_abi import GatedGrads
from stream_compaction_amd.sequence import _gated_args
from test_gpu_gated import inputs

pytestmark = pytest.mark.gpu

# That build's columns of 128 channels lose, in turn, the map of the walk's fourth tile, and the state at the border of
# its first 16 tiles.  Forward tiles have 128 tokens, the gradient's 64.
LOST = (4, 16)


def right_or_lost(got, want):
    lost = torch.isnan(got)
    assert torch.equal(got[~lost], want[~lost])
    return lost


@pytest.mark.parametrize("dt,d", [("f32", 256), ("bf16", 384), ("f32", 511)])
def test_words_that_never_come(dt, d):
    b, l = 3, 2610
    lengths = [2610, 2610, 200]                          # 21 and 41 tiles; the last has no lost word in the forward
    k, _, dy, dfinal = inputs((b, l, d, dt, lengths, "rate in"), 170, grads=True)
    parts = (d + 127) // 128
    y, state, starts = sc.gated_scan(keep_starts=True, **k)
    grads = sc.gated_scan_grad(dy, starts=starts, dfinal=dfinal, **k)
    assert not bool(torch.isnan(y).any()) and not bool(torch.isnan(grads["dx"]).any())

    L = sc.load(build.FALLBACK_LIB_PATH)
    a = _gated_args(k["x"], k["forget"], k["rate"], k["input_gate"], None, None, k["lengths"], False)
    y2, state2 = torch.empty_like(y), torch.empty_like(state)
    queue = torch.cuda.current_stream().cuda_stream
    scratch = torch.empty(L.gated_scan_scratch_bytes(a), dtype=torch.uint8, device="cuda")
    sc.check(L.gated_scan(a, y2.data_ptr(), state2.data_ptr(), None, scratch.data_ptr(), scratch.numel(), queue))
    torch.cuda.synchronize()
    lost = right_or_lost(y2, y)
    right_or_lost(state2, state)
    assert not bool(lost[:, :128].any()) and not bool(lost[2, 200:].any())
    for i in (0, 1):
        for part in range(parts):
            first = 128 * LOST[(i * parts + part) % 2]
            ch = slice(128 * part, min(d, 128 * part + 128))
            assert bool(lost[i, first:, ch].all()) and bool(torch.isnan(state2[i, ch]).all()), (i, part)

    g = {n: torch.empty_like(grads[n]) for n in ("dx", "dforget", "dinput_gate", "drate", "dstate")}
    p = {n: t.data_ptr() for n, t in g.items()}
    gs = GatedGrads(dy.data_ptr(), dy.stride()[:2], dfinal.data_ptr(), starts.data_ptr(), p["dx"], p["dforget"],
                    p["dinput_gate"], None, p["drate"], p["dstate"])
    scratch = torch.empty(L.gated_scan_grad_scratch_bytes(a), dtype=torch.uint8, device="cuda")
    sc.check(L.gated_scan_grad(a, gs, scratch.data_ptr(), scratch.numel(), queue))
    torch.cuda.synchronize()
    lost = {n: right_or_lost(g[n], grads[n]) for n in ("dx", "dforget", "dinput_gate", "dstate")}
    for i in (0, 1):
        # the walk begins with the last 50 tokens
        assert not bool(lost["dx"][i, 40 * 64:].any())
        for part in range(parts):
            last = 64 * (41 - LOST[(i * parts + part) % 2])
            ch = slice(128 * part, min(d, 128 * part + 128))
            assert bool(lost["dx"][i, :last, ch].all()) and bool(lost["dstate"][i, ch].all()), (i, part)
    assert bool(torch.isnan(g["drate"]).all())
