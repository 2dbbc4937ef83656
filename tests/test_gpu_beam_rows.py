"""Rows of states that one launch does not hold go out in several: in a build whose launches hold three workgroups, and at
the size where that happens in earnest."""
import ctypes

import numpy as np
import pytest
import torch

import beam_ref as ref
import stream_compaction_amd as sc
from stream_compaction_amd import build
from test_gpu_beam import raw, states_of
from test_gpu_sequence import gen

pytestmark = pytest.mark.gpu

# a workgroup moves 256 columns of 16 bytes (8 from 17 beams on, 4 from 33)
ROWS = [((7 * 4096 + 5,), "u8"), ((3,), "u8"), ((4096 * 3,), "u8"), ((4096 * 3 + 1,), "u8"), ((1024 * 5, 2), "f32"),
        ((0,), "f32"), ((4000,), "bf16")]


def move(L, states, parents, new_states):
    n, (b, k) = len(states), parents.shape
    size = [t.nbytes // (b * k) for t in states]
    status = L.beam_reorder((ctypes.c_void_p * n)(*[t.data_ptr() for t in states]),
                            (ctypes.c_void_p * n)(*[t.data_ptr() for t in new_states]), (ctypes.c_int64 * n)(*size), n,
                            parents.data_ptr(), b, k, torch.cuda.current_stream().cuda_stream)
    sc.check(status)
    torch.cuda.synchronize()


@pytest.mark.parametrize("b,k", [(1, 1), (2, 4), (3, 8), (1, 13), (2, 32), (1, 64)])
def test_rows_of_several_launches(b, k):
    L = sc.load(build.FALLBACK_LIB_PATH)
    g = gen(300 + k)
    p = torch.randint(0, k, (b, k), generator=g).int().cuda()
    for rows in ([ROWS[0]], ROWS):
        states = states_of(g, b, k, rows)
        want = [ref.reorder(raw(t, b, k), p.cpu().numpy()) for t in states]
        fresh = [torch.full_like(t, 3) for t in states]
        move(L, states, p, fresh)
        move(L, states, p, states)
        for i, (w, t, s) in enumerate(zip(want, fresh, states)):
            assert np.array_equal(raw(t, b, k), w), f"new {i}"
            assert np.array_equal(raw(s, b, k), w), f"in place {i}"


def test_rows_beyond_a_launch():
    # two beams of 64 GiB change places: 2^24 workgroups
    n = (64 << 30) + 40
    free, _ = torch.cuda.mem_get_info()
    if free < 2 * n + (8 << 30):
        pytest.skip("needs 136 GiB of GPU memory")
    big = torch.zeros((1, 2, n), dtype=torch.uint8, device="cuda")
    places = [0, (32 << 30) - 4096, 32 << 30, (48 << 30) + 12345, (64 << 30) - 100, n - 1000]
    for i, at in enumerate(places):
        big[0, 0, at:at + 1000], big[0, 1, at:at + 1000] = 2 * i + 1, 2 * i + 2
    want = [[big[0, j, at - min(at, 2000):at + 3000].clone() for j in (1, 0)] for at in places]
    sc.beam_reorder([big], torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"))
    for at, pair in zip(places, want):
        for j in (0, 1):
            assert torch.equal(big[0, j, at - min(at, 2000):at + 3000], pair[j]), (at, j)
    del big
    torch.cuda.empty_cache()
