"""Sizes whose products pass 64 bits are refused, on the host: nothing is launched (no GPU here, and
the pointers are fake addresses)."""
import ctypes

import stream_compaction_amd as sc
from stream_compaction_amd._sequence_abi import ConvArgs, ScanArgs, ScanGrads

EINVAL = 1
S = [0x10000000 * (i + 1) for i in range(24)]
BIG = 1 << 30                      # BIG tokens of BIG sequences x 16 channels: 2^64 elements


def conv_args(batch, length, channels):
    a = ConvArgs(x=S[0], weight=S[1], batch=batch, length=length, channels=channels, width=1,
                 dtype=sc.DTYPE_CODES["bf16"])
    return a                       # strides of 0: x itself is one token


def scan_args(batch, length, channels, states=1):
    return ScanArgs(x=S[0], dt=S[1], B=S[2], C=S[3], A=S[5], batch=batch, length=length,
                    channels=channels, states=states, groups=1, dtype=sc.DTYPE_CODES["bf16"])


def test_token_counts_past_64_bits():
    L = sc.lib()
    stride = (ctypes.c_int64 * 2)(0, 0)
    for batch, length, channels in ((BIG, BIG, 16), (BIG, BIG, 48), (1 << 26, BIG, 1 << 20)):
        a = conv_args(batch, length, channels)
        assert L.causal_conv(a, S[5], None, None) == EINVAL
        assert L.causal_conv_grad_scratch_bytes(a) == 0
        assert L.causal_conv_grad(a, S[4], stride, None, S[6], S[7], None, None, S[8], 1 << 46,
                                  None) == EINVAL
        s = scan_args(batch, length, channels)
        assert L.selective_scan(s, S[10], None, None, None) == EINVAL
        assert L.selective_scan_split(s, S[10], None, None, S[11], 1 << 46, None) == EINVAL
        for size in ("starts", "split_scratch", "grad_scratch"):
            assert getattr(L, f"selective_scan_{size}_bytes")(s) == 0
        g = ScanGrads(dy=S[10], starts=S[12], dx=S[13], ddt=S[14], dB=S[15], dC=S[16], dA=S[18])
        assert L.selective_scan_grad(s, g, S[19], 1 << 46, None) == EINVAL


def test_starts_of_2_to_the_47_bytes():
    # 2^45 bytes of activations, 2^48 of kept states
    L = sc.lib()
    s = scan_args(1 << 17, 1 << 17, 1 << 10, 64)
    assert L.selective_scan(s, S[10] << 20, None, S[12], None) == EINVAL
