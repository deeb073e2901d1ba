"""ctypes declarations of include/gdr.h and the loader of libgdr.so."""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

GDR_OK, GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED, GDR_ERR_ALIGNMENT = 0, 1, 2, 3
GDR_ERR_WORKSPACE, GDR_ERR_CUDA, GDR_ERR_DEVICE_CHECK, GDR_ERR_TIMEOUT = 4, 5, 6, 7
GDR_ERR_RANGE = 8
F32, BF16 = 0, 1
READ_POST, READ_PRE = 0, 1
WRITE_PLAIN, WRITE_GATE, WRITE_TIED = 0, 1, 2
ACT_NONE, ACT_SILU, ACT_SIGMOID = 0, 1, 2

# every symbol include/gdr.h declares
EXPORTS = ["gdr_chunk_fwd_workspace_size", "gdr_chunk_fwd", "gdr_chunk_fwd_noalloc",
           "gdr_noalloc_read_device_error",
           "gdr_chunk_bwd_workspace_size", "gdr_chunk_bwd",
           "gdr_chunk_fwd_bidir_workspace_size", "gdr_chunk_fwd_bidir",
           "gdr_chunk_fwd_path", "gdr_chunk_bwd_path",
           "gdr_decode_step", "gdr_status_string", "gdr_read_device_error", "gdr_version",
           "gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step",
           "gdr_conv_fwd", "gdr_conv_bwd_workspace_size", "gdr_conv_bwd", "gdr_conv_step",
           "gdr_norm_fwd_workspace_size", "gdr_norm_fwd",
           "gdr_norm_bwd_workspace_size", "gdr_norm_bwd"]


class ChunkArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hk", ctypes.c_int),
                ("Hv", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("n_seqs", ctypes.c_int), ("chunk", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("read_mode", ctypes.c_int),
                ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
                ("reverse", ctypes.c_int), ("o_accumulate", ctypes.c_int),
                ("gate_raw", ctypes.c_int), ("gate_A", ctypes.c_void_p),
                ("gate_dt_bias", ctypes.c_void_p), ("beta_scale", ctypes.c_float),
                ("gdn2", ctypes.c_int), ("gdn2_w", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("read_mode", ctypes.c_int),
                ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
                ("gate_raw", ctypes.c_int), ("gate_A", ctypes.c_void_p),
                ("gate_dt_bias", ctypes.c_void_p), ("beta_scale", ctypes.c_float),
                ("out_norm", ctypes.c_int), ("norm_z", ctypes.c_void_p),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
                ("gdn2", ctypes.c_int), ("gdn2_w", ctypes.c_void_p)]


class ScanArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("n_seqs", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("write", ctypes.c_int),
                ("reverse", ctypes.c_int), ("status", ctypes.c_void_p)]


class ConvArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("n_seqs", ctypes.c_int), ("width", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("reverse", ctypes.c_int),
                ("status", ctypes.c_void_p)]


class NormArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("d", ctypes.c_int), ("n_seqs", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("per_sequence", ctypes.c_int), ("center", ctypes.c_int),
                ("activation", ctypes.c_int), ("shared_weight", ctypes.c_int),
                ("eps", ctypes.c_float), ("status", ctypes.c_void_p)]


class GdrError(RuntimeError):
    def __init__(self, status: int, msg: str = ""):
        self.status = status
        super().__init__(msg or status_string(status))


_lock = threading.Lock()
_lib = None


def _declare(lib):
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.gdr_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(ChunkArgs)]
    lib.gdr_chunk_fwd_workspace_size.restype = sz
    lib.gdr_chunk_fwd.argtypes = [ctypes.POINTER(ChunkArgs)] + [vp] * 10 + [sz, vp]
    lib.gdr_chunk_fwd.restype = ctypes.c_int
    lib.gdr_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkArgs)] + [vp] * 10
    lib.gdr_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.gdr_noalloc_read_device_error.argtypes = [vp]
    lib.gdr_noalloc_read_device_error.restype = ctypes.c_int
    lib.gdr_chunk_fwd_bidir_workspace_size.argtypes = [ctypes.POINTER(ChunkArgs)]
    lib.gdr_chunk_fwd_bidir_workspace_size.restype = sz
    lib.gdr_chunk_fwd_bidir.argtypes = [ctypes.POINTER(ChunkArgs)] + [vp] * 10 + [sz, vp]
    lib.gdr_chunk_fwd_bidir.restype = ctypes.c_int
    lib.gdr_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(ChunkArgs)]
    lib.gdr_chunk_bwd_workspace_size.restype = sz
    lib.gdr_chunk_bwd.argtypes = [ctypes.POINTER(ChunkArgs)] + [vp] * 16 + [sz, vp]
    lib.gdr_chunk_bwd.restype = ctypes.c_int
    lib.gdr_chunk_fwd_path.argtypes = [ctypes.POINTER(ChunkArgs)]
    lib.gdr_chunk_fwd_path.restype = ctypes.c_char_p
    lib.gdr_chunk_bwd_path.argtypes = [ctypes.POINTER(ChunkArgs)]
    lib.gdr_chunk_bwd_path.restype = ctypes.c_char_p
    lib.gdr_decode_step.argtypes = [ctypes.POINTER(DecodeArgs)] + [vp] * 8
    lib.gdr_decode_step.restype = ctypes.c_int
    lib.gdr_status_string.argtypes = [ctypes.c_int]
    lib.gdr_status_string.restype = ctypes.c_char_p
    lib.gdr_read_device_error.argtypes = [ctypes.POINTER(ChunkArgs), vp, vp]
    lib.gdr_read_device_error.restype = ctypes.c_int
    for name, args, n, ws in (
            ("gdr_scan_fwd", ScanArgs, 7, False), ("gdr_scan_bwd", ScanArgs, 12, False),
            ("gdr_scan_step", ScanArgs, 6, False), ("gdr_conv_fwd", ConvArgs, 7, False),
            ("gdr_conv_bwd", ConvArgs, 11, True), ("gdr_conv_step", ConvArgs, 6, False),
            ("gdr_norm_fwd", NormArgs, 8, True), ("gdr_norm_bwd", NormArgs, 12, True)):
        f = getattr(lib, name)  # args, n pointers (the workspace's size behind it), the stream
        f.argtypes = [ctypes.POINTER(args)] + [vp] * n + ([sz] if ws else []) + [vp]
        f.restype = ctypes.c_int
    for name, args in (("gdr_conv_bwd", ConvArgs), ("gdr_norm_fwd", NormArgs),
                       ("gdr_norm_bwd", NormArgs)):
        f = getattr(lib, name + "_workspace_size")
        f.argtypes = [ctypes.POINTER(args)]
        f.restype = sz
    lib.gdr_version.argtypes = []
    lib.gdr_version.restype = ctypes.c_char_p
    return lib


def lib():
    """Load libgdr.so once.  Raises FileNotFoundError if it has not been built: there is
    no fallback implementation."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise FileNotFoundError(
                    f"{LIB_PATH} is missing; build it with "
                    "`python -m gated_delta_rule_146_b200.build`")
            _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().gdr_status_string(int(status)).decode()
    except FileNotFoundError:
        return f"gdr status {status}"


def check(status: int):
    if status != GDR_OK:
        raise GdrError(status)
