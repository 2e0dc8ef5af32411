"""ctypes binding of libqvg's C ABI (include/qvg.h), with the same names.

This module only marshals arguments: every step of the compression path runs in the CUDA
kernels of libqvg.so.  There is no fallback; if the library is missing or does not load,
every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libqvg.so")

QVG_OK = 0
QVG_ERR_INVALID_ARG = 1
QVG_ERR_UNSUPPORTED = 2
QVG_ERR_WORKSPACE = 3
QVG_ERR_CUDA = 4
QVG_ERR_DEVICE = 5
QVG_ERR_SCRATCH_LIMIT = 6
QVG_STATIC_SCRATCH_BYTES = 64 << 20

QVG_DEV_NONFINITE = 0x1
QVG_DEV_TIMEOUT = 0x2
QVG_DEV_BAD_INDEX = 0x4
QVG_DEV_NO_PAGES = 0x8
QVG_FEW_SEQS = 1024

QVG_F16, QVG_BF16, QVG_F32 = 0, 1, 2
QVG_QSCHEME_SYMMETRIC, QVG_QSCHEME_MIDRISE = 0, 1
QVG_STEP_PLANES, QVG_STEP_GEMM, QVG_STEP_REFINE = 1, 2, 4
QVG_CENTROIDS_F32, QVG_CENTROIDS_F16, QVG_CENTROIDS_BF16 = 0, 1, 2
QVG_PAGE_F16, QVG_PAGE_BF16, QVG_PAGE_E4M3, QVG_PAGE_INT8 = 0, 1, 2, 3
QVG_PAGE_E2M1, QVG_PAGE_INT4 = 8, 9


class qvg_quant_params(ctypes.Structure):
    _fields_ = [
        ("n_tensors", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("C", ctypes.c_int32),
        ("T", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("iters", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32),
        ("seed", ctypes.c_uint64),
        ("tensor_id_base", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("token_offset", ctypes.c_int64),
        ("token_capacity", ctypes.c_int64),
        ("table_index", ctypes.c_int32),
        ("n_tables", ctypes.c_int32),
        ("warm_stride", ctypes.c_int64),
        ("qscheme", ctypes.c_int32),
        ("centroid_format", ctypes.c_int32),
    ]


class qvg_buffers(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("pi", ctypes.c_void_p),
        ("centroids", ctypes.c_void_p),
    ]


class qvg_dequant_params(ctypes.Structure):
    _fields_ = [
        ("n_tensors", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("C", ctypes.c_int32),
        ("T", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("chunk_len", ctypes.c_int64),
        ("token_capacity", ctypes.c_int64),
        ("n_tables", ctypes.c_int32),
        ("out_stride", ctypes.c_int64),
        ("qscheme", ctypes.c_int32),
    ]


class qvg_attention_params(ctypes.Structure):
    _fields_ = [
        ("n_heads", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("M", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("C", ctypes.c_int32),
        ("T", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("qscheme", ctypes.c_int32),
        ("chunk_len", ctypes.c_int64),
        ("token_capacity", ctypes.c_int64),
        ("n_tables", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("k_first", ctypes.c_int64),
        ("v_first", ctypes.c_int64),
        ("tensor_step", ctypes.c_int64),
    ]


class qvg_pages(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("k_group", ctypes.c_void_p),
        ("v_group", ctypes.c_void_p),
    ]


class qvg_rotary(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("n_axes", ctypes.c_int32),
        ("sections", ctypes.c_int32 * 4),
        ("mscale", ctypes.c_float),
        ("pos_stride", ctypes.c_int64),
        ("positions", ctypes.c_void_p),
        ("freqs", ctypes.c_void_p),
    ]


class qvg_rope_params(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64),
        ("n_heads", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("backward", ctypes.c_int32),
        ("x_token_stride", ctypes.c_int64),
        ("x_head_stride", ctypes.c_int64),
        ("y_token_stride", ctypes.c_int64),
        ("y_head_stride", ctypes.c_int64),
    ]


class qvg_page_write_params(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64),
        ("n_heads", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("n_pages", ctypes.c_int64),
        ("in_dtype", ctypes.c_int32),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
    ]


class qvg_page_read_params(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("n_pages", ctypes.c_int64),
        ("max_pages", ctypes.c_int32),
        ("first", ctypes.c_int64),
        ("count", ctypes.c_int64),
        ("x_seq_stride", ctypes.c_int64),
        ("x_tensor_stride", ctypes.c_int64),
    ]


class qvg_page_attention_params(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("n_pages", ctypes.c_int64),
        ("max_pages", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("window", ctypes.c_int64),
        ("total_q", ctypes.c_int64),
        ("max_q", ctypes.c_int64),
        ("max_kv", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("o_token_stride", ctypes.c_int64),
        ("o_head_stride", ctypes.c_int64),
    ]


class qvg_page_table_params(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("n_pages", ctypes.c_int64),
        ("total", ctypes.c_int64),
        ("out_pages", ctypes.c_int64),
        ("starts", ctypes.c_void_p),
    ]


# Every symbol include/qvg.h declares, with its ctypes signature.
SIGNATURES = {
    "qvg_quantize_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(qvg_quant_params)]),
    "qvg_quantize": (ctypes.c_int, [ctypes.POINTER(qvg_quant_params), ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.POINTER(qvg_buffers),
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                     ctypes.c_void_p]),
    "qvg_quantize_static": (ctypes.c_int, [ctypes.POINTER(qvg_quant_params), ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.POINTER(qvg_buffers),
                                            ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_reassign": (ctypes.c_int, [ctypes.POINTER(qvg_quant_params), ctypes.c_void_p,
                                    ctypes.POINTER(qvg_buffers), ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_reassign_steps": (ctypes.c_int, [ctypes.POINTER(qvg_quant_params), ctypes.c_void_p,
                                          ctypes.POINTER(qvg_buffers), ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "qvg_selftest_assign_timeout": (ctypes.c_int, [ctypes.POINTER(qvg_quant_params),
                                                   ctypes.c_void_p, ctypes.POINTER(qvg_buffers),
                                                   ctypes.c_void_p, ctypes.c_size_t,
                                                   ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_dequantize": (ctypes.c_int, [ctypes.POINTER(qvg_dequant_params),
                                      ctypes.POINTER(qvg_buffers), ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_attention_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(qvg_attention_params)]),
    "qvg_attention": (ctypes.c_int, [ctypes.POINTER(qvg_attention_params), ctypes.c_void_p,
                                     ctypes.POINTER(qvg_buffers), ctypes.POINTER(qvg_buffers),
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_rope": (ctypes.c_int, [ctypes.POINTER(qvg_rope_params), ctypes.POINTER(qvg_rotary),
                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_write": (ctypes.c_int, [ctypes.POINTER(qvg_page_write_params), ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.POINTER(qvg_rotary), ctypes.POINTER(qvg_pages),
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_read": (ctypes.c_int, [ctypes.POINTER(qvg_page_read_params),
                                     ctypes.POINTER(qvg_pages), ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_attention_workspace_bytes": (ctypes.c_size_t,
                                           [ctypes.POINTER(qvg_page_attention_params)]),
    "qvg_page_attention": (ctypes.c_int, [ctypes.POINTER(qvg_page_attention_params),
                                          ctypes.c_void_p, ctypes.POINTER(qvg_pages),
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_table_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(qvg_page_table_params)]),
    "qvg_page_copy": (ctypes.c_int, [ctypes.POINTER(qvg_page_table_params), ctypes.c_int64,
                                     ctypes.POINTER(qvg_pages), ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.POINTER(qvg_pages), ctypes.c_int64,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_append": (ctypes.c_int, [ctypes.POINTER(qvg_page_table_params),
                                       ctypes.POINTER(qvg_pages), ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_fork": (ctypes.c_int, [ctypes.POINTER(qvg_page_table_params),
                                     ctypes.POINTER(qvg_pages), ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                     ctypes.c_void_p]),
    "qvg_page_free": (ctypes.c_int, [ctypes.POINTER(qvg_page_table_params), ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qvg_page_compact": (ctypes.c_int, [ctypes.POINTER(qvg_page_table_params),
                                        ctypes.POINTER(qvg_pages), ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.POINTER(qvg_pages),
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "qvg_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qvg_version": (ctypes.c_uint32, []),
}

_lock = threading.Lock()
_lib = None


class QVGError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s failed: %s (status %d)" % (what, qvg_status_string(code)
                                                        if _lib is not None else "?", code))


def load(path: str | None = None):
    """Load libqvg.so (once).  Raises if it is missing: there is no fallback path."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libqvg.so not found at %s; build it with "
                               "video_kv_cache_gb300.build.build()" % p)
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _ref(obj):
    return ctypes.byref(obj) if obj is not None else None


def qvg_quantize_workspace_bytes(params: qvg_quant_params) -> int:
    return int(load().qvg_quantize_workspace_bytes(_ref(params)))


def qvg_quantize(params: qvg_quant_params, X: int, warm_centroids: int | None,
                 out: qvg_buffers, workspace: int, workspace_bytes: int,
                 dev_status: int | None, stream: int | None) -> int:
    return int(load().qvg_quantize(_ref(params), X, warm_centroids, _ref(out),
                                   workspace, workspace_bytes, dev_status, stream))


def qvg_quantize_static(params: qvg_quant_params, X: int, warm_centroids: int | None,
                        out: qvg_buffers, dev_status: int | None, stream: int | None) -> int:
    return int(load().qvg_quantize_static(_ref(params), X, warm_centroids, _ref(out),
                                          dev_status, stream))


def qvg_reassign(params: qvg_quant_params, X: int, out: qvg_buffers, workspace: int,
                 workspace_bytes: int, dev_status: int | None, stream: int | None) -> int:
    return int(load().qvg_reassign(_ref(params), X, _ref(out), workspace, workspace_bytes,
                                   dev_status, stream))


def qvg_reassign_steps(params: qvg_quant_params, X: int, out: qvg_buffers, workspace: int,
                       workspace_bytes: int, steps: int, dev_status: int | None,
                       stream: int | None) -> int:
    return int(load().qvg_reassign_steps(_ref(params), X, _ref(out), workspace, workspace_bytes,
                                         steps, dev_status, stream))


def qvg_selftest_assign_timeout(params: qvg_quant_params, X: int, out: qvg_buffers,
                                workspace: int, workspace_bytes: int, dev_status: int | None,
                                stream: int | None) -> int:
    return int(load().qvg_selftest_assign_timeout(_ref(params), X, _ref(out), workspace,
                                                  workspace_bytes, dev_status, stream))


def qvg_dequantize(params: qvg_dequant_params, inp: qvg_buffers, X_hat: int,
                   dev_status: int | None, stream: int | None) -> int:
    return int(load().qvg_dequantize(_ref(params), _ref(inp), X_hat,
                                     dev_status, stream))


def qvg_attention_workspace_bytes(params: qvg_attention_params) -> int:
    return int(load().qvg_attention_workspace_bytes(_ref(params)))


def qvg_attention(params: qvg_attention_params, Q: int, k_cache: qvg_buffers,
                  v_cache: qvg_buffers, O: int, workspace: int | None, workspace_bytes: int,
                  dev_status: int | None, stream: int | None) -> int:
    return int(load().qvg_attention(_ref(params), Q, _ref(k_cache), _ref(v_cache), O,
                                    workspace, workspace_bytes, dev_status, stream))


def qvg_rope(params: qvg_rope_params, rotary: qvg_rotary, X: int, Y: int,
             stream: int | None) -> int:
    return (_lib or load()).qvg_rope(_ref(params), _ref(rotary), X, Y, stream)


def qvg_page_write(params: qvg_page_write_params, K: int, V: int, slots: int,
                   rotary: qvg_rotary | None, pages: qvg_pages, dev_status: int | None,
                   stream: int | None) -> int:
    return (_lib or load()).qvg_page_write(_ref(params), K, V, slots, _ref(rotary), _ref(pages),
                                           dev_status, stream)


def qvg_page_read(params: qvg_page_read_params, pages: qvg_pages, page_table: int,
                  seq_lens: int, X: int, dev_status: int | None, stream: int | None) -> int:
    return (_lib or load()).qvg_page_read(_ref(params), _ref(pages), page_table, seq_lens, X,
                                          dev_status, stream)


def qvg_page_attention_workspace_bytes(params: qvg_page_attention_params) -> int:
    return (_lib or load()).qvg_page_attention_workspace_bytes(_ref(params))


def qvg_page_attention(params: qvg_page_attention_params, Q: int, pages: qvg_pages,
                       page_table: int, seq_lens: int, cu_q: int | None, O: int,
                       lse: int | None, workspace: int | None, workspace_bytes: int,
                       dev_status: int | None, stream: int | None) -> int:
    return (_lib or load()).qvg_page_attention(_ref(params), Q, _ref(pages), page_table, seq_lens,
                                               cu_q, O, lse, workspace, workspace_bytes, dev_status,
                                               stream)


def qvg_page_table_workspace_bytes(params: qvg_page_table_params) -> int:
    return (_lib or load()).qvg_page_table_workspace_bytes(_ref(params))


def qvg_page_copy(params: qvg_page_table_params, n: int, pages: qvg_pages, src: int, dst: int,
                  rows: int | None, to: qvg_pages, to_pages: int, dev_status: int | None,
                  stream: int | None) -> int:
    return (_lib or load()).qvg_page_copy(_ref(params), n, _ref(pages), src, dst, rows, _ref(to),
                                          to_pages, dev_status, stream)


def qvg_page_append(params: qvg_page_table_params, pages: qvg_pages, refs: int, page_table: int,
                    seq_lens: int, counts: int, slots: int | None, positions: int | None,
                    copies: int, workspace: int, workspace_bytes: int, dev_status: int | None,
                    stream: int | None) -> int:
    return (_lib or load()).qvg_page_append(_ref(params), _ref(pages), refs, page_table, seq_lens,
                                            counts, slots, positions, copies, workspace,
                                            workspace_bytes, dev_status, stream)


def qvg_page_fork(params: qvg_page_table_params, pages: qvg_pages, refs: int, page_table: int,
                  seq_lens: int, parents: int, copies: int, workspace: int, workspace_bytes: int,
                  dev_status: int | None, stream: int | None) -> int:
    return (_lib or load()).qvg_page_fork(_ref(params), _ref(pages), refs, page_table, seq_lens,
                                          parents, copies, workspace, workspace_bytes, dev_status,
                                          stream)


def qvg_page_free(params: qvg_page_table_params, refs: int, page_table: int, seq_lens: int,
                  drop_first: int | None, drop_last: int | None, dev_status: int | None,
                  stream: int | None) -> int:
    return (_lib or load()).qvg_page_free(_ref(params), refs, page_table, seq_lens, drop_first,
                                          drop_last, dev_status, stream)


def qvg_page_compact(params: qvg_page_table_params, pages: qvg_pages, refs: int, page_table: int,
                     seq_lens: int, to: qvg_pages, out_table: int, out_refs: int, live: int,
                     workspace: int, workspace_bytes: int, dev_status: int | None,
                     stream: int | None) -> int:
    return (_lib or load()).qvg_page_compact(_ref(params), _ref(pages), refs, page_table, seq_lens,
                                             _ref(to), out_table, out_refs, live, workspace,
                                             workspace_bytes, dev_status, stream)


def qvg_status_string(code: int) -> str:
    return load().qvg_status_string(code).decode()


def qvg_version() -> int:
    return int(load().qvg_version())
