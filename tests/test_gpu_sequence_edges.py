"""The sequence operators at their edges on the GPU: batches that go out as several launches."""
import pytest
import torch

import stream_compaction_amd as sc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [13, 16])
def test_scan_step_over_several_launches(n):
    # a launch takes 2^21 workgroups of 256 lanes: here an odd number of sequences (299593),
    # two to a lane; the sequences at its end move once, in place as into a new state
    d = {13: 112, 16: 385}[n]
    lanes = d * (16 if n == 13 else 4)
    step = (1 << 21) // ((lanes + 255) // 256)
    b = step + 2
    assert step % 2 == 1
    r = torch.Generator(device="cuda").manual_seed(n)
    one = lambda *shape: torch.randn(shape, generator=r, device="cuda")  # noqa: E731
    x, dt = (one(1, d).bfloat16().expand(b, d) for _ in range(2))
    B, C = (one(b, 1, n).bfloat16() for _ in range(2))
    A, D = -torch.rand((d, n), generator=r, device="cuda"), one(d)
    state = one(1, d, n).expand(b, d, n).contiguous()
    first = state[0].clone()
    fresh = torch.empty_like(state)
    y = sc.selective_scan_step(state, x, dt, A, B, C, D, softplus=True, new_state=fresh)
    y2 = sc.selective_scan_step(state, x, dt, A, B, C, D, softplus=True)
    assert torch.equal(y, y2) and torch.equal(state, fresh)
    for i in (0, 1, step - 2, step - 1, step, step + 1):
        s = slice(i, i + 1)
        new = torch.empty((1, d, n), device="cuda")
        v = sc.selective_scan_step(first[None].clone(), x[s], dt[s], A, B[s], C[s], D,
                                   softplus=True, new_state=new)
        assert torch.equal(v, y[s]) and torch.equal(new[0], state[i]), f"sequence {i}"
    del state, fresh
    torch.cuda.empty_cache()
