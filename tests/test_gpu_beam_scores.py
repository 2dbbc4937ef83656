"""Scores of beam selection are 64-bit ones, and equal scores are equal to the bit: certain tokens whatever their
logit, rows that are one another plus a constant, ended beams beside certain ones, tails beside a sure token.
Choices and ties against the float64 oracle of ``beam_ref``."""
import math

import numpy as np
import pytest
import torch

import beam_ref as ref
import stream_compaction_amd as sc
from test_gpu_sequence import TYPES, gen

pytestmark = pytest.mark.gpu
INF = float("inf")

# A row's sum of exponentials relative to its maximum is off by its roundings in 64 bits: at most 64 terms a lane,
# 6 steps over lanes, 3 over waves and one a segment (below 64 here) in order, each 2^-53 of the sum, and the
# exponentials' own 5e-16 < 2^-50; its logarithm by as much, absolutely, and a score of size below 32 by three roundings of
# 2^-53 x 32 more: (64 + 6 + 3 + 64) 2^-53 + 2^-50 + 96 x 2^-53 < 2^-44.
IN_64_BITS = 2.0 ** -44


def check(x, scores, count, finished=None, end=0):
    f = None if finished is None else finished.cuda()
    got = sc.beam_select(x, scores.cuda(), count, finished=f, end_token=end)
    want = ref.select(x.double().cpu().numpy(), scores.double().numpy(), count,
                      None if finished is None else finished.numpy(), end)
    assert np.array_equal(got[1].cpu().numpy(), want[1]), "parents"
    assert np.array_equal(got[2].cpu().numpy(), want[2]), "tokens"
    a, b = got[0].double().cpu().numpy(), want[0]
    low = np.isinf(b)
    assert np.array_equal(a[low], b[low]), "infinite scores"
    assert (np.abs(a[~low] - b[~low]) <= np.abs(b[~low]) * 2.0 ** -24 + IN_64_BITS).all(), "scores"
    return got


VALUES = [7.25, 0.0, 1.0, -20.0, 30.0, 599.0, 601.0, -601.0]


@pytest.mark.parametrize("v", [3, 2048, 20011, 50000])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_certain_tokens(dt, v):
    # one token a beam has a chance, at another place and of another logit in each: all have their beam's score
    places = [v - 1, 0, v // 2, v // 3, 1, v - 2, v // 2 + 1, 2]
    x = torch.full((2, 8, v), -INF)
    for j in range(8):
        x[:, j, places[j]] = VALUES[j]
    x = x.to(TYPES[dt]).cuda()
    scores = torch.full((2, 8), -1.375)
    scores[1] = torch.tensor([-3.0, -2.0, -2.0, -3.0, -2.5, -2.0, -2.5, -3.0])
    for n in (1, 2, 8, 16):
        got = check(x, scores, n)
        n = min(n, 8)
        assert got[1][0, :n].tolist() == list(range(n))
        assert got[0][0, :n].tolist() == [-1.375] * n
        assert got[0][1, :n].tolist() == sorted(scores[1].tolist(), reverse=True)[:n]
    # every second beam has ended, at the same score
    done = torch.tensor([[0, 1] * 4, [1, 0] * 4], dtype=torch.uint8)
    for n in (1, 8):
        got = check(x, torch.full((2, 8), -1.375), n, done, v // 2)
        assert got[1].tolist() == [list(range(n))] * 2 and got[0].tolist() == [[-1.375] * n] * 2


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_two_tokens_lie_anywhere(dt):
    # two tokens have a chance, with the same difference and in other places in each beam
    v = 33001
    pairs = [(5, 30000), (32999, 4), (100, 101), (20000, 9000), (0, 33000), (12345, 12344)]
    x = torch.full((1, 6, v), -INF)
    for j, (a, b) in enumerate(pairs):
        x[0, j, a], x[0, j, b] = 10.0 * j - 20, 10.0 * j - 23
    got = check(x.to(TYPES[dt]).cuda(), torch.zeros(1, 6), 12)
    assert got[1][0].tolist() == list(range(6)) * 2
    assert got[2][0].tolist() == [a for a, _ in pairs] + [b for _, b in pairs]


@pytest.mark.parametrize("v", [9, 4099, 40003])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_rows_that_differ_by_a_constant(dt, v):
    # a constant that every logit takes up exactly: all beams' scores are equal, and the lower beam goes first
    g = gen(60 + v)
    if dt == "f32":
        row = torch.randint(-2048, 2049, (2, 1, v), generator=g) / 256.0
        shift = torch.tensor([0.25, 0.0, -7.0, 33.5, 595.0, -700.0, 1000.0, 12.0])
    else:
        row = torch.randint(-7, 8, (2, 1, v), generator=g).float()
        shift = torch.tensor([1.0, 0.0, -7.0, 33.0, 100.0, -100.0, 120.0, 5.0])
    wide = row + shift[:, None]
    x = wide.to(TYPES[dt])
    assert torch.equal(x.float(), wide)
    for n in (1, 8, 9, 64):
        got = check(x.cuda(), torch.full((2, 8), -0.5), n)
        m = min(n, 8)
        # (a beam may have its greatest logit more than once)
        assert bool((got[1][:, :m].diff(dim=1) >= 0).all()) and bool((got[0][:, :m] == got[0][:, :1]).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_sure_token_among_others(dt):
    # the log probability is what the others leave: -(v - 1) exp(-top)
    v = 50000
    for top in (12.0, 20.0, 24.0, 28.0, 32.0, 36.0):
        for base in (0.0, 16.0):
            x = torch.full((1, 2, v), base)
            x[0, 0, 31000], x[0, 1, 7] = base + top, base + top
            got = sc.beam_select(x.to(TYPES[dt]).cuda(), torch.zeros(1, 2, device="cuda"), 2)
            # (two sums of the same terms in another order: either beam may be a last bit ahead)
            assert sorted(zip(got[1][0].tolist(), got[2][0].tolist())) == [(0, 31000), (1, 7)]
            want = -math.log1p((v - 1) * math.exp(-top))
            assert float((got[0].double() - want).abs().max()) <= abs(want) * 2.0 ** -24 + IN_64_BITS, (top, base)
            assert float(got[0].max()) <= 0.0


def test_scores_that_cancel():
    # a beam's own score that takes its best token's away leaves the digits behind float32's
    g = gen(61)
    x = torch.randn((3, 4, 30011), generator=g) * 3
    lp = np.stack([[ref.log_softmax(x[i, j].numpy()) for j in range(4)] for i in range(3)])
    scores = torch.tensor(-lp.max(-1)).float()
    check(x.cuda(), scores, 4)
