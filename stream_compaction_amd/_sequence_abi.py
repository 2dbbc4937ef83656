"""ctypes mirror of the sequence operators in ``include/scan.h`` (needs no torch)."""
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


def declare(L):
    """C signatures of the sequence entry points on a loaded library."""
    sz, f32 = ctypes.c_size_t, ctypes.c_float
    conv, scan = ctypes.POINTER(ConvArgs), ctypes.POINTER(ScanArgs)
    for name, args in (
            ("causal_conv", [conv, _vp, _vp, _vp]),
            ("causal_conv_grad", [conv, _vp, ctypes.POINTER(_i64), _vp, _vp, _vp, _vp, _vp, _vp,
                                  sz, _vp]),
            ("causal_conv_step", [conv, _vp, _vp, _vp, _vp]),
            ("selective_scan", [scan, _vp, _vp, _vp, _vp]),
            ("selective_scan_split", [scan, _vp, _vp, _vp, _vp, sz, _vp]),
            ("selective_scan_grad", [scan, ctypes.POINTER(ScanGrads), _vp, sz, _vp]),
            ("selective_scan_step", [scan, _vp, _vp, _vp, _vp]),
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
                       ("embedding_grad_scratch_bytes", [_i64, _i64, _i64])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = sz
