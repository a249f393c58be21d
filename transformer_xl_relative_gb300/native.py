"""ctypes declarations of libtxl.so (the C ABI in include/txl.h).

Argument marshalling only.  There is no fallback: if the library is missing the import of the
binding raises, and every non-OK status of a call raises ``TxlError``.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
# TXL_CHECKED=1 selects the range-checked build of the same library (built on request by
# _build.py --checked)
LIB_PATH = os.path.join(_HERE, "libtxl_checked.so" if os.environ.get("TXL_CHECKED") == "1" else "libtxl.so")

TXL_OK, TXL_ERR_INVALID_ARG, TXL_ERR_UNSUPPORTED, TXL_ERR_ALIGNMENT = 0, 1, 2, 3
TXL_ERR_CUDA, TXL_ERR_TIMEOUT, TXL_ERR_WORKSPACE, TXL_ERR_PAGE = 4, 5, 6, 7
TXL_F32, TXL_BF16 = 0, 1

# every function include/txl.h declares
EXPORTS = (
    "txl_status_str", "txl_version", "txl_rel_pos_gen", "txl_rel_attn_fwd",
    "txl_rel_attn_workspace_size", "txl_rel_attn_path", "txl_rel_attn_decode",
    "txl_rel_attn_decode_workspace_size", "txl_rel_attn_decode_noalloc", "txl_mem_push",
    "txl_selftest_wait_timeout", "txl_linear", "txl_rel_attn_layer", "txl_rel_attn_layer_workspace_size",
    "txl_rel_attn_layer_fused", "txl_rel_attn_layer_fused_workspace_size",
    "txl_checked_build", "txl_range_errors", "txl_range_errors_clear", "txl_selftest_range_check",
    "txl_rel_attn_bwd", "txl_rel_attn_bwd_workspace_size", "txl_rel_pos_bwd", "txl_rel_attn_table_fwd",
    "txl_rel_attn_table_path", "txl_rel_attn_decode_path", "txl_rel_attn_fwd_lse", "txl_rel_attn_bwd_lse",
    "txl_rel_attn_bwd_path", "txl_qmem_row_bytes", "txl_qmem_push", "txl_qmem_read",
    "txl_rel_attn_qmem", "txl_rel_attn_qmem_workspace_size", "txl_rel_attn_qmem_path",
    "txl_rel_attn_qmem_call", "txl_qmem_push_call", "txl_qmem_read_call",
    "txl_paged_push", "txl_rel_attn_paged", "txl_rel_attn_paged_workspace_size", "txl_paged_evict",
    "txl_paged_evict_workspace_size", "txl_q4_bytes", "txl_q4_quantise", "txl_q4_expand", "txl_linear_q4",
    "txl_linear_q4_workspace_size", "txl_paged_push_call", "txl_linear_q4_call",
)


class TxlView(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class TxlMem(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("stride_h", ctypes.c_int64),
                ("B", ctypes.c_int), ("M", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("wp", ctypes.c_int), ("valid", ctypes.c_int)]


class TxlQmem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p),
                ("B", ctypes.c_int), ("M", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("bits", ctypes.c_int), ("wp", ctypes.c_int), ("valid", ctypes.c_int)]


class TxlPaged(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "pos", "weight", "table", "length", "next_pos", "scratch",
                                               "err_flag")] + \
               [(n, ctypes.c_int) for n in ("B", "H", "D", "ld", "n_pages", "page_len", "max_pages", "dtype")]


class TxlQ4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("k", ctypes.c_int), ("n", ctypes.c_int), ("group", ctypes.c_int)]


# txl_rel_attn_paged_args: T, clamp_len, n_rows, accumulate, scale; mem; the views q, k_new, v_new, out; counts, u,
# v_bias, r, ld_r, workspace, workspace_bytes, stream (pointers as unsigned 64-bit numbers)
PAGED_ARGS = struct.Struct("@4if" + "Q" + 4 * "Qqqq" + "QQQQqQQQ")
# txl_paged_push_args: mem; the views k_new, v_new; counts, stream; T
PAGED_PUSH_ARGS = struct.Struct("@Q" + 2 * "Qqqq" + "QQi")
# txl_linear_q4_args: w, X, ld_x, Y, ld_y, workspace, workspace_bytes, err_flag, stream, m
Q4_ARGS = struct.Struct("@QQqQqQQQQi")
# txl_qmem_kv_args: mem; the views k, v; j0, n, dtype; stream (pointers as unsigned 64-bit numbers)
QMEM_KV_ARGS = struct.Struct("@Q" + 2 * "Qqqq" + "3iQ")
# txl_rel_attn_qmem_args: B, L, H, D, clamp_len, n_rows, dtype, scale; the views q, k_cur, v_cur, out; mem, u,
# v_bias, r, ld_r, workspace, workspace_bytes, err_flag, stream (pointers as unsigned 64-bit numbers)
QMEM_ARGS = struct.Struct("@7if" + 4 * "Qqqq" + "QQQQqQQQQ")


class TxlError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, status_str(status), status))


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libtxl.so once.  Raises ImportError when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libtxl.so is not built (expected at %s); run "
                          "`python -c \"import __graft_entry__ as g; g.build()\"`" % path)
    lib = ctypes.CDLL(path)
    V = ctypes.POINTER(TxlView)
    Mp = ctypes.POINTER(TxlMem)
    i, i64, vp, fp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    lib.txl_status_str.argtypes = [i]
    lib.txl_status_str.restype = ctypes.c_char_p
    lib.txl_version.argtypes = []
    lib.txl_version.restype = i
    lib.txl_rel_pos_gen.argtypes = [i, i, i, i, vp, i64, vp, i64, i, vp]
    lib.txl_rel_pos_gen.restype = i
    lib.txl_rel_attn_fwd.argtypes = [i, i, i, i, i, V, Mp, V, V, vp, vp, vp, i64, i, fp, V, i,
                                     vp, ctypes.c_size_t, vp, vp]
    lib.txl_rel_attn_fwd.restype = i
    lib.txl_rel_attn_workspace_size.argtypes = [i, i, i, i, Mp, i]
    lib.txl_rel_attn_workspace_size.restype = ctypes.c_size_t
    lib.txl_rel_attn_path.argtypes = [i, i, i, i, V, Mp, V, V, vp, i64, V, i]
    lib.txl_rel_attn_path.restype = i
    lib.txl_rel_attn_decode.argtypes = [i, i, i, i, i, V, Mp, V, V, vp, vp, vp, i64, i, fp, V, i,
                                        vp, ctypes.c_size_t, vp]
    lib.txl_rel_attn_decode.restype = i
    lib.txl_rel_attn_decode_workspace_size.argtypes = [i, i, i, i, Mp]
    lib.txl_rel_attn_decode_workspace_size.restype = ctypes.c_size_t
    lib.txl_rel_attn_decode_noalloc.argtypes = [i, i, i, i, i, V, Mp, V, V, vp, vp, vp, i64, i, fp, V,
                                                i, vp]
    lib.txl_rel_attn_decode_noalloc.restype = i
    lib.txl_mem_push.argtypes = [Mp, V, V, i, vp]
    lib.txl_mem_push.restype = i
    lib.txl_checked_build.argtypes = []
    lib.txl_checked_build.restype = i
    lib.txl_range_errors.argtypes = [ctypes.POINTER(ctypes.c_int)]
    lib.txl_range_errors.restype = i
    lib.txl_range_errors_clear.argtypes = []
    lib.txl_range_errors_clear.restype = i
    lib.txl_selftest_range_check.argtypes = [vp]
    lib.txl_selftest_range_check.restype = i
    lib.txl_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint, vp]
    lib.txl_selftest_wait_timeout.restype = i
    lib.txl_linear.argtypes = [i, i, i, vp, i64, vp, i64, vp, i64, i, vp, vp]
    lib.txl_linear.restype = i
    lib.txl_rel_attn_layer.argtypes = [i, i, i, i, i, i, vp, i64, Mp, vp, vp, vp, vp, vp, i64, i, fp,
                                       vp, i64, vp, ctypes.c_size_t, vp, vp]
    lib.txl_rel_attn_layer.restype = i
    lib.txl_rel_attn_layer_workspace_size.argtypes = [i, i, i, i]
    lib.txl_rel_attn_layer_workspace_size.restype = ctypes.c_size_t
    lib.txl_rel_attn_layer_fused.argtypes = [i, i, i, i, i, i, vp, i64, Mp, i, vp, vp, vp, vp, vp, i64, i, fp,
                                             vp, i64, vp, ctypes.c_size_t, vp, vp]
    lib.txl_rel_attn_layer_fused.restype = i
    lib.txl_rel_attn_layer_fused_workspace_size.argtypes = [i, i, i, i]
    lib.txl_rel_attn_layer_fused_workspace_size.restype = ctypes.c_size_t
    lib.txl_rel_attn_bwd.argtypes = [i, i, i, i, i, V, Mp, V, V, vp, vp, vp, i64, i, fp, V, V,
                                     vp, vp, vp, vp, vp, vp, i, vp, ctypes.c_size_t, vp]
    lib.txl_rel_attn_bwd.restype = i
    lib.txl_rel_attn_fwd_lse.argtypes = [i, i, i, i, i, V, Mp, V, V, vp, vp, vp, i64, i, fp, V, vp, i,
                                         vp, ctypes.c_size_t, vp, vp]
    lib.txl_rel_attn_fwd_lse.restype = i
    lib.txl_rel_attn_bwd_lse.argtypes = [i, i, i, i, i, V, Mp, V, V, vp, vp, vp, i64, i, fp, V, V, vp,
                                         vp, vp, vp, vp, vp, vp, i, vp, ctypes.c_size_t, vp]
    lib.txl_rel_attn_bwd_lse.restype = i
    lib.txl_rel_attn_bwd_path.argtypes = [i, i, i, i, V, Mp, V, V, vp, i64, V, V, vp, vp, vp, vp, i]
    lib.txl_rel_attn_bwd_path.restype = i
    lib.txl_rel_attn_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.txl_rel_attn_bwd_workspace_size.restype = ctypes.c_size_t
    lib.txl_rel_pos_bwd.argtypes = [i, i, i, i, vp, vp, i64, vp]
    lib.txl_rel_pos_bwd.restype = i
    lib.txl_rel_attn_table_fwd.argtypes = [i, i, i, i, i, V, V, V, vp, vp, vp, i64, vp, fp, V, i, vp]
    lib.txl_rel_attn_table_fwd.restype = i
    lib.txl_rel_attn_table_path.argtypes = [i, i, i, i, i, V, V, V, vp, i64, vp, V, i]
    lib.txl_rel_attn_table_path.restype = i
    lib.txl_rel_attn_decode_path.argtypes = [i, i, i, i, V, Mp, V, V, vp, i64, V, i]
    lib.txl_rel_attn_decode_path.restype = i
    Qp = ctypes.POINTER(TxlQmem)
    lib.txl_qmem_row_bytes.argtypes = [i, i]
    lib.txl_qmem_row_bytes.restype = ctypes.c_size_t
    lib.txl_qmem_push.argtypes = [Qp, V, V, i, i, vp]
    lib.txl_qmem_push.restype = i
    lib.txl_qmem_read.argtypes = [Qp, i, i, V, V, i, vp]
    lib.txl_qmem_read.restype = i
    lib.txl_rel_attn_qmem.argtypes = [i, i, i, i, i, V, Qp, V, V, vp, vp, vp, i64, i, fp, V, i,
                                      vp, ctypes.c_size_t, vp, vp]
    lib.txl_rel_attn_qmem.restype = i
    lib.txl_rel_attn_qmem_call.argtypes = [ctypes.c_char_p]
    lib.txl_rel_attn_qmem_call.restype = i
    lib.txl_qmem_push_call.argtypes = [ctypes.c_char_p]
    lib.txl_qmem_push_call.restype = i
    lib.txl_qmem_read_call.argtypes = [ctypes.c_char_p]
    lib.txl_qmem_read_call.restype = i
    lib.txl_rel_attn_qmem_workspace_size.argtypes = [i, i, i, i, Qp, i]
    lib.txl_rel_attn_qmem_workspace_size.restype = ctypes.c_size_t
    lib.txl_rel_attn_qmem_path.argtypes = [i, i, i, i, V, Qp, V, V, vp, i64, V, i]
    lib.txl_rel_attn_qmem_path.restype = i
    Pp, Wp, sz = ctypes.POINTER(TxlPaged), ctypes.POINTER(TxlQ4), ctypes.c_size_t
    lib.txl_paged_push.argtypes = [Pp, V, V, i, vp, vp]
    lib.txl_paged_push.restype = i
    lib.txl_paged_push_call.argtypes = [ctypes.c_char_p]
    lib.txl_paged_push_call.restype = i
    lib.txl_linear_q4_call.argtypes = [ctypes.c_char_p]
    lib.txl_linear_q4_call.restype = i
    lib.txl_rel_attn_paged.argtypes = [ctypes.c_char_p]
    lib.txl_rel_attn_paged.restype = i
    lib.txl_rel_attn_paged_workspace_size.argtypes = [Pp, i, i, i]
    lib.txl_rel_attn_paged_workspace_size.restype = sz
    lib.txl_paged_evict.argtypes = [Pp, i, i, vp, sz, vp]
    lib.txl_paged_evict.restype = i
    lib.txl_paged_evict_workspace_size.argtypes = [Pp]
    lib.txl_paged_evict_workspace_size.restype = sz
    lib.txl_q4_bytes.argtypes = [i, i, i]
    lib.txl_q4_bytes.restype = sz
    lib.txl_q4_quantise.argtypes = [Wp, vp, i64, vp]
    lib.txl_q4_quantise.restype = i
    lib.txl_q4_expand.argtypes = [Wp, vp, i64, vp]
    lib.txl_q4_expand.restype = i
    lib.txl_linear_q4.argtypes = [i, Wp, vp, i64, vp, i64, vp, sz, vp, vp]
    lib.txl_linear_q4.restype = i
    lib.txl_linear_q4_workspace_size.argtypes = [i, Wp]
    lib.txl_linear_q4_workspace_size.restype = sz
    _lib = lib
    return lib


def status_str(status: int) -> str:
    try:
        return load().txl_status_str(int(status)).decode()
    except ImportError:
        return "status %d" % status


def check(status: int, what: str) -> None:
    if status != TXL_OK:
        raise TxlError(status, what)
