"""ctypes mirror of the sequence operators and of beam search in ``include/scan.h`` (needs no torch)."""
import ctypes

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class ConvArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("weight", _vp), ("bias", _vp), ("initial_state", _vp),
                ("lengths", _vp), ("batch", _i64), ("length", _i64), ("channels", _i64),
                ("width", _i64), ("x_stride", _i64 * 2), ("silu", _i32), ("dtype", _i32)]


class ScanArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("dt", _vp), ("B", _vp), ("C", _vp), ("z", _vp), ("A", _vp),
                ("D", _vp), ("dt_bias", _vp), ("initial_state", _vp), ("lengths", _vp),
                ("batch", _i64), ("length", _i64), ("channels", _i64), ("states", _i64),
                ("groups", _i64), ("x_stride", _i64 * 2), ("dt_stride", _i64 * 2),
                ("z_stride", _i64 * 2), ("B_stride", _i64 * 3), ("C_stride", _i64 * 3),
                ("softplus", _i32), ("dtype", _i32)]


class ScanGrads(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dy_stride", _i64 * 2), ("dfinal", _vp), ("starts", _vp),
                ("dx", _vp), ("ddt", _vp), ("dB", _vp), ("dC", _vp), ("dz", _vp), ("dA", _vp),
                ("dD", _vp), ("ddt_bias", _vp), ("dinitial", _vp)]


# (strides one by one: a step for one token is bound by this side, and arrays cost more)
class GatedArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("forget", _vp), ("input_gate", _vp), ("z", _vp), ("rate", _vp),
                ("initial_state", _vp), ("lengths", _vp), ("batch", _i64), ("length", _i64),
                ("channels", _i64), ("x_batch", _i64), ("x_token", _i64), ("forget_batch", _i64),
                ("forget_token", _i64), ("input_gate_batch", _i64), ("input_gate_token", _i64),
                ("z_batch", _i64), ("z_token", _i64), ("dtype", _i32)]


class GatedGrads(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dy_stride", _i64 * 2), ("dfinal", _vp), ("starts", _vp),
                ("dx", _vp), ("dforget", _vp), ("dinput_gate", _vp), ("dz", _vp), ("drate", _vp),
                ("dinitial", _vp)]


class BeamArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("scores", _vp), ("finished", _vp), ("batch", _i64),
                ("beams", _i64), ("vocab", _i64), ("count", _i64), ("end_token", _i64),
                ("logits_batch", _i64), ("logits_beam", _i64), ("dtype", _i32)]


def declare(L):
    """C signatures of the sequence entry points on a loaded library."""
    sz, f32 = ctypes.c_size_t, ctypes.c_float
    conv, scan = ctypes.POINTER(ConvArgs), ctypes.POINTER(ScanArgs)
    gated, beam = ctypes.POINTER(GatedArgs), ctypes.POINTER(BeamArgs)
    for name, args in (
            ("causal_conv", [conv, _vp, _vp, _vp]),
            ("causal_conv_grad", [conv, _vp, ctypes.POINTER(_i64), _vp, _vp, _vp, _vp, _vp, _vp,
                                  sz, _vp]),
            ("causal_conv_step", [conv, _vp, _vp, _vp, _vp]),
            ("selective_scan", [scan, _vp, _vp, _vp, _vp]),
            ("selective_scan_split", [scan, _vp, _vp, _vp, _vp, sz, _vp]),
            ("selective_scan_grad", [scan, ctypes.POINTER(ScanGrads), _vp, sz, _vp]),
            ("selective_scan_step", [scan, _vp, _vp, _vp, _vp]),
            ("gated_scan", [gated, _vp, _vp, _vp, _vp, sz, _vp]),
            ("gated_scan_grad", [gated, ctypes.POINTER(GatedGrads), _vp, sz, _vp]),
            ("gated_scan_step", [gated, _vp, _vp, _vp, _vp]),
            ("beam_select", [beam, _vp, _vp, _vp, _vp, sz, _vp]),
            ("beam_reorder", [_vp, _vp, _vp, _i64, _vp, _i64, _i64, _vp]),
            ("embedding", [_vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, f32,
                           _vp]),
            ("embedding_grad", [_vp, _vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                ctypes.c_int, f32, _vp, sz, _vp])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    for name, args in (("causal_conv_grad_scratch_bytes", [conv]),
                       ("selective_scan_starts_bytes", [scan]),
                       ("selective_scan_split_scratch_bytes", [scan]),
                       ("selective_scan_grad_scratch_bytes", [scan]),
                       ("gated_scan_starts_bytes", [gated]),
                       ("gated_scan_scratch_bytes", [gated]),
                       ("gated_scan_grad_scratch_bytes", [gated]),
                       ("beam_select_scratch_bytes", [beam]),
                       ("embedding_grad_scratch_bytes", [_i64, _i64, _i64])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = sz
