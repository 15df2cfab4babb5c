"""ctypes loader and signatures of libdiffattn.so (include/diffattn.h)."""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdiffattn.so")

DIFFATTN_OK = 0
DIFFATTN_ERR_INVALID = -1
DIFFATTN_ERR_UNSUPPORTED = -2
DIFFATTN_ERR_CUDA = -3
DIFFATTN_ERR_TIMEOUT = -4
DIFFATTN_ERR_INDEX = -5

DIFFATTN_BF16 = 0
DIFFATTN_F32 = 1

DIFFATTN_KERNEL_TCGEN05 = 1
DIFFATTN_KERNEL_SIMT = 2

DIFFATTN_MAX_AXES = 4

DIFFATTN_NORM_NONE = 0
DIFFATTN_NORM_RMS = 1
DIFFATTN_NORM_GROUP = 2

# Every symbol include/diffattn.h declares.
EXPORTED = (
    "diffattn_lambda",
    "diffattn_lambda_backward",
    "diffattn_fwd",
    "diffattn_fwd_ex",
    "diffattn_fwd_host",
    "diffattn_fwd_train",
    "diffattn_bwd",
    "diffattn_bwd_saved",
    "diffattn_bwd_workspace_bytes",
    "diffattn_decode",
    "diffattn_decode_workspace_bytes",
    "diffattn_decode_noalloc",
    "diffattn_workspace_bytes",
    "diffattn_rotary",
    "diffattn_rotary_bwd",
    "diffattn_rotary_bwd_workspace_bytes",
    "diffattn_rotary_axes",
    "diffattn_rotary_axes_bwd",
    "diffattn_paged_append",
    "diffattn_paged_append_axes",
    "diffattn_paged_decode",
    "diffattn_paged_workspace_bytes",
    "diffattn_cross_fwd",
    "diffattn_cross_fwd_ex",
    "diffattn_cross_workspace_bytes",
    "diffattn_cross_bwd",
    "diffattn_cross_bwd_ex",
    "diffattn_cross_bwd_workspace_bytes",
    "diffattn_head_norm",
    "diffattn_head_norm_bwd",
    "diffattn_head_norm_bwd_workspace_bytes",
    "diffattn_select_kernel",
    "diffattn_get_device_error",
    "diffattn_selftest_timeout",
    "diffattn_strerror",
    "diffattn_version",
)


class DiffattnDesc(ctypes.Structure):
    """Mirror of diffattn_desc."""
    _fields_ = [
        ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("kv_group", ctypes.c_int32),
        ("q1_stride", ctypes.c_int64 * 3), ("k1_stride", ctypes.c_int64 * 3),
        ("q2_stride", ctypes.c_int64 * 3), ("k2_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3), ("o_stride", ctypes.c_int64 * 3),
        ("Dv", ctypes.c_int64),
    ]


class DiffattnKvDesc(ctypes.Structure):
    """Mirror of diffattn_kv_desc."""
    _fields_ = [
        ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("Tq", ctypes.c_int64), ("Tk", ctypes.c_int64),
        ("D", ctypes.c_int64), ("dtype", ctypes.c_int32), ("kv_group", ctypes.c_int32),
        ("q1_stride", ctypes.c_int64 * 3), ("k1_stride", ctypes.c_int64 * 3),
        ("q2_stride", ctypes.c_int64 * 3), ("k2_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3), ("o_stride", ctypes.c_int64 * 3),
        ("Dv", ctypes.c_int64),
    ]


class DiffattnEpilogue(ctypes.Structure):
    """Mirror of diffattn_epilogue."""
    _fields_ = [
        ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("out_scale", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


class DiffattnRotaryDesc(ctypes.Structure):
    """Mirror of diffattn_rotary_desc."""
    _fields_ = [
        ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int64), ("H", ctypes.c_int64),
        ("Hk", ctypes.c_int64), ("dtype", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
        ("pos64", ctypes.c_int32), ("table_rows", ctypes.c_int64), ("pos_stride", ctypes.c_int64 * 2),
        ("q_weight_stride", ctypes.c_int64), ("k_weight_stride", ctypes.c_int64),
        ("q1_stride", ctypes.c_int64 * 3), ("k1_stride", ctypes.c_int64 * 3),
        ("q2_stride", ctypes.c_int64 * 3), ("k2_stride", ctypes.c_int64 * 3),
        ("q1_grad_stride", ctypes.c_int64 * 3), ("k1_grad_stride", ctypes.c_int64 * 3),
        ("q2_grad_stride", ctypes.c_int64 * 3), ("k2_grad_stride", ctypes.c_int64 * 3),
    ]


class DiffattnAxes(ctypes.Structure):
    """Mirror of diffattn_axes."""
    _fields_ = [
        ("n", ctypes.c_int32), ("pairs", ctypes.c_int32 * DIFFATTN_MAX_AXES), ("reserved", ctypes.c_int32),
        ("pos_stride", ctypes.c_int64),
    ]


class DiffattnPages(ctypes.Structure):
    """Mirror of diffattn_pages."""
    _fields_ = [
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("max_pages", ctypes.c_int64),
        ("block_table_stride", ctypes.c_int64), ("k1_stride", ctypes.c_int64 * 3),
        ("k2_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
    ]


class DiffattnPagedDesc(ctypes.Structure):
    """Mirror of diffattn_paged_desc."""
    _fields_ = [
        ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("Tq", ctypes.c_int64), ("D", ctypes.c_int64),
        ("Dv", ctypes.c_int64), ("dtype", ctypes.c_int32), ("kv_group", ctypes.c_int32),
        ("q1_stride", ctypes.c_int64 * 3), ("q2_stride", ctypes.c_int64 * 3),
        ("o_stride", ctypes.c_int64 * 3), ("mask_stride", ctypes.c_int64 * 2),
        ("zero_rest", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class DiffattnCrossDesc(ctypes.Structure):
    """Mirror of diffattn_cross_desc."""
    _fields_ = [
        ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("Tq", ctypes.c_int64), ("Tk", ctypes.c_int64),
        ("D", ctypes.c_int64), ("Dv", ctypes.c_int64), ("dtype", ctypes.c_int32), ("kv_group", ctypes.c_int32),
        ("lambda_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("q1_stride", ctypes.c_int64 * 3), ("k1_stride", ctypes.c_int64 * 3),
        ("q2_stride", ctypes.c_int64 * 3), ("k2_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3), ("o_stride", ctypes.c_int64 * 3), ("dout_stride", ctypes.c_int64 * 3),
    ]


class DiffattnNormDesc(ctypes.Structure):
    """Mirror of diffattn_norm_desc."""
    _fields_ = [
        ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("T", ctypes.c_int64), ("C", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("out_scale", ctypes.c_float),
        ("x_stride", ctypes.c_int64 * 3), ("y_stride", ctypes.c_int64 * 3),
        ("dy_stride", ctypes.c_int64 * 3), ("dx_stride", ctypes.c_int64 * 3),
    ]


class DiffattnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.diffattn_lambda.argtypes = [vp, vp, vp, vp, i64, ctypes.c_double, vp, vp]
    lib.diffattn_lambda.restype = ctypes.c_int
    lib.diffattn_lambda_backward.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp]
    lib.diffattn_lambda_backward.restype = ctypes.c_int
    lib.diffattn_fwd.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp, ctypes.c_float,
                                 vp, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    lib.diffattn_fwd_ex.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp, ctypes.c_float,
                                    vp, ctypes.c_int, ctypes.POINTER(DiffattnEpilogue), vp, vp,
                                    ctypes.c_size_t, vp]
    lib.diffattn_fwd_ex.restype = ctypes.c_int
    lib.diffattn_decode.argtypes = [ctypes.POINTER(DiffattnKvDesc), vp, vp, vp, vp, vp, ctypes.c_float,
                                    vp, ctypes.c_int, ctypes.POINTER(DiffattnEpilogue), vp, vp,
                                    ctypes.c_size_t, vp]
    lib.diffattn_decode.restype = ctypes.c_int
    lib.diffattn_decode_noalloc.argtypes = [ctypes.POINTER(DiffattnKvDesc), vp, vp, vp, vp, vp,
                                            ctypes.c_float, vp, ctypes.c_int,
                                            ctypes.POINTER(DiffattnEpilogue), vp, vp]
    lib.diffattn_decode_noalloc.restype = ctypes.c_int
    lib.diffattn_bwd.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp, ctypes.c_float,
                                 vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.diffattn_bwd.restype = ctypes.c_int
    lib.diffattn_fwd_host.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp,
                                      ctypes.c_float, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp,
                                      vp, ctypes.c_size_t, vp]
    lib.diffattn_fwd_host.restype = ctypes.c_int
    lib.diffattn_fwd_train.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp,
                                       ctypes.c_float, vp, ctypes.c_int, vp, vp, vp, vp,
                                       ctypes.c_size_t, vp]
    lib.diffattn_fwd_train.restype = ctypes.c_int
    lib.diffattn_bwd_saved.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp,
                                       ctypes.c_float, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.diffattn_bwd_saved.restype = ctypes.c_int
    lib.diffattn_bwd_workspace_bytes.argtypes = [ctypes.POINTER(DiffattnDesc)]
    lib.diffattn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.diffattn_decode_workspace_bytes.argtypes = [ctypes.POINTER(DiffattnKvDesc)]
    lib.diffattn_decode_workspace_bytes.restype = ctypes.c_size_t
    # (called from csrc/binding.cpp; here for tests of the ABI)
    lib.diffattn_rotary.argtypes = [vp] * 15
    lib.diffattn_rotary.restype = ctypes.c_int
    lib.diffattn_rotary_bwd.argtypes = [vp] * 21 + [ctypes.c_size_t, vp]
    lib.diffattn_rotary_bwd.restype = ctypes.c_int
    lib.diffattn_rotary_bwd_workspace_bytes.argtypes = [vp]
    lib.diffattn_rotary_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.diffattn_paged_append.argtypes = [vp, i64] + [vp] * 16
    lib.diffattn_paged_append.restype = ctypes.c_int
    lib.diffattn_rotary_axes.argtypes = [vp] * 16
    lib.diffattn_rotary_axes.restype = ctypes.c_int
    lib.diffattn_rotary_axes_bwd.argtypes = [vp] * 22 + [ctypes.c_size_t, vp]
    lib.diffattn_rotary_axes_bwd.restype = ctypes.c_int
    lib.diffattn_paged_append_axes.argtypes = [vp, vp, i64] + [vp] * 16
    lib.diffattn_paged_append_axes.restype = ctypes.c_int
    lib.diffattn_paged_decode.argtypes = [vp] * 11 + [ctypes.c_float, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.diffattn_paged_decode.restype = ctypes.c_int
    lib.diffattn_paged_workspace_bytes.argtypes = [vp, vp]
    lib.diffattn_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.diffattn_cross_fwd.argtypes = [vp] * 7 + [ctypes.c_float] + [vp] * 6 + [ctypes.c_size_t, vp]
    lib.diffattn_cross_fwd.restype = ctypes.c_int
    lib.diffattn_cross_bwd.argtypes = [vp] * 7 + [ctypes.c_float] + [vp] * 12 + [ctypes.c_size_t, vp]
    lib.diffattn_cross_bwd.restype = ctypes.c_int
    lib.diffattn_cross_fwd_ex.argtypes = [vp] * 7 + [ctypes.c_float] + [vp] * 7 + [ctypes.c_size_t, vp]
    lib.diffattn_cross_fwd_ex.restype = ctypes.c_int
    lib.diffattn_cross_bwd_ex.argtypes = [vp] * 7 + [ctypes.c_float] + [vp] * 13 + [ctypes.c_size_t, vp]
    lib.diffattn_cross_bwd_ex.restype = ctypes.c_int
    for f in (lib.diffattn_cross_workspace_bytes, lib.diffattn_cross_bwd_workspace_bytes):
        f.argtypes = [vp]
        f.restype = ctypes.c_size_t
    lib.diffattn_head_norm.argtypes = [vp] * 6
    lib.diffattn_head_norm.restype = ctypes.c_int
    lib.diffattn_head_norm_bwd.argtypes = [vp] * 8 + [ctypes.c_size_t, vp]
    lib.diffattn_head_norm_bwd.restype = ctypes.c_int
    lib.diffattn_head_norm_bwd_workspace_bytes.argtypes = [vp]
    lib.diffattn_head_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.diffattn_workspace_bytes.argtypes = []
    lib.diffattn_workspace_bytes.restype = ctypes.c_size_t
    lib.diffattn_fwd.restype = ctypes.c_int
    lib.diffattn_select_kernel.argtypes = [ctypes.POINTER(DiffattnDesc), vp, vp, vp, vp, vp, vp]
    lib.diffattn_select_kernel.restype = ctypes.c_int
    lib.diffattn_get_device_error.argtypes = [vp]
    lib.diffattn_get_device_error.restype = ctypes.c_int
    lib.diffattn_selftest_timeout.argtypes = [vp]
    lib.diffattn_selftest_timeout.restype = ctypes.c_int
    lib.diffattn_strerror.argtypes = [ctypes.c_int]
    lib.diffattn_strerror.restype = ctypes.c_char_p
    lib.diffattn_version.argtypes = []
    lib.diffattn_version.restype = ctypes.c_int
    _lib = lib
    return lib


def strerror(code: int) -> str:
    try:
        return load().diffattn_strerror(code).decode()
    except RuntimeError:
        return f"error {code}"


def check(code: int, what: str) -> None:
    if code != DIFFATTN_OK:
        raise DiffattnError(code, what)
