"""Sizes that beam search refuses before anything is launched (no GPU needed)."""
import ctypes

import stream_compaction_amd as sc

EINVAL = 1


def test_rows_too_long_to_count():
    # in fewer than 2^47 bytes in all, but more workgroups than 32 bits count
    L, at = sc.lib(), ctypes.c_void_p * 1
    for size in (1 << 43, (1 << 46) + 3):
        for to in (1 << 12, 1 << 46):
            assert L.beam_reorder(at(1 << 12), at(to), (ctypes.c_int64 * 1)(size), 1, 1 << 47, 1, 1, None) == EINVAL, size
