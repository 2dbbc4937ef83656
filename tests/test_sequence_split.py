"""The split scan's entry points refuse what they must (needs no GPU: nothing is launched)."""
import ctypes

import stream_compaction_amd as sc
from stream_compaction_amd._sequence_abi import ScanArgs, ScanGrads

EINVAL, ENOTSUP, EALIAS, ESCRATCH = 1, 2, 3, 4
S = [0x10000000 * (i + 1) for i in range(16)]


def args(batch=1, length=4096, channels=64, states=16, groups=1):
    a = ScanArgs(*S[:10])
    a.lengths = a.initial_state = None
    a.batch, a.length, a.channels, a.states, a.groups = batch, length, channels, states, groups
    for name in ("x_stride", "dt_stride", "z_stride"):
        getattr(a, name)[:] = (length * channels, channels)
    a.B_stride[:] = a.C_stride[:] = (length * groups * states, groups * states, states)
    a.softplus, a.dtype = 1, sc.DTYPE_CODES["f32"]
    return a


def test_scratch_sizes():
    need = sc.lib().selective_scan_split_scratch_bytes
    # chunks of 128 tokens at least, (states + 1) float32 per chunk and channel
    size = need(args())
    chunks = size // (64 * 17 * 4)
    assert size == chunks * 64 * 17 * 4 and 2 <= chunks <= 32
    # a short scan, or one whose channels fill the card, is not split
    assert need(args(length=300)) == 0 and need(args(channels=4096)) == 0
    assert need(args(batch=0)) == 0 and need(args(length=0)) == 0 and need(args(states=65)) == 0
    # what the gradient asks for grows with it
    grad = sc.lib().selective_scan_grad_scratch_bytes
    part = 4 * 4096 * 2 * 16 * 4
    assert grad(args()) == part + chunks * 64 * 18 * 4 + size


def test_refusals():
    L = sc.lib()
    a = args()
    need = L.selective_scan_split_scratch_bytes(a)

    def call(a=a, y=S[10], fs=S[11], starts=None, scratch=S[12], room=need):
        return L.selective_scan_split(a, y, fs, starts, scratch, room, None)
    assert call(room=need - 1) == ESCRATCH and call(scratch=None) == EINVAL
    assert call(scratch=S[12] + 8) == EINVAL and call(y=None) == EINVAL
    assert call(scratch=S[0]) == EALIAS and call(scratch=S[10]) == EALIAS
    assert call(y=S[0]) == EALIAS and call(starts=S[12]) == EALIAS
    assert call(a=args(states=65)) == ENOTSUP and call(a=args(groups=3)) == EINVAL
    assert L.selective_scan_split(ctypes.POINTER(ScanArgs)(), S[10], S[11], None, S[12], need, None) == EINVAL
    g = ScanGrads()
    assert L.selective_scan_grad(a, g, S[12], 1 << 40, None) == EINVAL
