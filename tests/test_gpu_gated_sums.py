"""The gradient by the rate adds up what many sequences give without losing digits."""
import pytest
import torch

import stream_compaction_amd as sc
from test_gpu_sequence import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("l", [1, 70])
@pytest.mark.parametrize("b", [4096, 65536])
def test_rate_gradient_of_equal_sequences(b, l):
    # every sequence gives the same terms: the sum is one sequence's times a power of two, exactly but for each
    # side's rounding to float32 (2^-24 of it)
    d = 37
    g = gen(200 + l)
    x, f, i, dy = (torch.randn((1, l, d), generator=g).cuda().expand(b, l, d) for _ in range(4))
    rate = (0.05 + torch.rand(d, generator=g)).cuda()
    one = [t[:1].contiguous() for t in (x, f, i, dy)]
    _, _, starts = sc.gated_scan(one[0], one[1], rate, one[2], keep_starts=True)
    want = sc.gated_scan_grad(one[3], one[0], one[1], starts, rate, one[2])["drate"].double() * b
    _, _, starts = sc.gated_scan(x, f, rate, i, keep_starts=True)
    got = sc.gated_scan_grad(dy, x, f, starts, rate, i)["drate"].double()
    assert bool(torch.isfinite(want).all()) and float(want.abs().min()) > 0
    assert bool(((got - want).abs() <= 2 * 2.0 ** -24 * want.abs()).all())
