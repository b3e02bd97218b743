"""Python binding of libqsa.so, the C-ABI QSA hot path for B200 (sm_100a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind ``include/qsa.h``.  PyTorch supplies device memory and the
current stream.  The entry points keep the C names (``qsa_prefill`` ...)
and take torch tensors; bf16 data may be ``torch.bfloat16`` or ``torch.uint16``
(bit patterns).  If libqsa.so is missing this module raises on first use:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqsa.so")
LIB_DEBUG_PATH = os.path.join(_PKG, "libqsa_debug.so")   # the debug build (tests of the failure handling)

QSA_OK = 0
_STATUS = {0: "QSA_OK", 1: "QSA_ERR_INVALID_ARG", 2: "QSA_ERR_UNSUPPORTED", 3: "QSA_ERR_MISALIGNED",
           4: "QSA_ERR_WORKSPACE_TOO_SMALL", 5: "QSA_ERR_CUDA", 6: "QSA_ERR_DEVICE_TIMEOUT",
           7: "QSA_ERR_DEVICE_BOUNDS", 8: "QSA_ERR_ARCH"}

EXPORTED = ["qsa_default_params", "qsa_status_string", "qsa_last_error", "qsa_index_scores", "qsa_select_blocks",
            "qsa_select_workspace_size", "qsa_prefill", "qsa_prefill_workspace_size", "qsa_decode",
            "qsa_decode_workspace_size", "qsa_check_device_error", "qsa_trace_begin", "qsa_trace_end",
            "qsa_decode_noalloc", "qsa_prefill_cached", "qsa_prefill_cached_workspace_size",
            "qsa_index_workspace_size", "qsa_decode_mean_pool", "qsa_mean_pool_keys",
            "qsa_decode_reuse", "qsa_verify", "qsa_verify_workspace_size", "qsa_set_decode_splits",
            "qsa_decode_noalloc_check_error", "qsa_default_layer_params", "qsa_norm_rope", "qsa_paged_append",
            "qsa_paged_decode", "qsa_paged_prefill", "qsa_paged_workspace_size"]

KERNEL_NAMES = {1: "rope_table", 2: "rope_k", 3: "indexer", 4: "select", 5: "attention", 6: "decode_append",
                7: "decode_indexer", 8: "decode_attention", 9: "decode_combine",
                10: "mean_pool_keys", 11: "verify_expand", 12: "idx_rope", 13: "norm_rope", 14: "paged_append",
                15: "paged_decode", 16: "paged_decode_join", 17: "paged_prefill", 18: "paged_prefill_join"}


class QSAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}" + (f" ({detail})" if detail else ""))


class qsa_params(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("rope_theta", ctypes.c_double), ("idx_heads", ctypes.c_int32),
                ("idx_dim", ctypes.c_int32), ("block_size", ctypes.c_int32), ("budget_blocks", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("aggregation", ctypes.c_int32),
                ("yarn_factor", ctypes.c_double), ("yarn_original_max", ctypes.c_double),
                ("yarn_beta_fast", ctypes.c_double), ("yarn_beta_slow", ctypes.c_double),
                ("idx_rope", ctypes.c_int32)]


class qsa_layer_params(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("rope_axes", ctypes.c_int32),
                ("rope_section", ctypes.c_int32 * 3), ("rope_interleaved", ctypes.c_int32),
                ("rope_theta", ctypes.c_double), ("yarn_factor", ctypes.c_double),
                ("yarn_original_max", ctypes.c_double), ("yarn_beta_fast", ctypes.c_double),
                ("yarn_beta_slow", ctypes.c_double), ("norm_eps", ctypes.c_float),
                ("norm_zero_centred", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("window", ctypes.c_int32),
                ("n_sinks", ctypes.c_int32)]


class qsa_paged_kv(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("table_ld", ctypes.c_int64)]


# element types of the paged-cache calls (qsa_layer_params.dtype)
DTYPE_BF16 = 0
DTYPE_FP16 = 1

# block-score aggregation (qsa_params.aggregation)
AGG_TOKEN_MAX = 0
AGG_MEAN_POOL = 1

_lib = None


_libs: dict = {}
_lib_path = None


def load(path: str = LIB_PATH):
    """Load libqsa.so and declare its signatures (raises if it is not built).
    The first library loaded serves every call of this module (see
    use_library)."""
    global _lib, _lib_path
    if _lib is not None:
        return _lib
    _lib = _open(path)
    _lib_path = path
    return _lib


def use_library(path: str) -> str | None:
    """Route this module's calls to the library at ``path`` (e.g. the debug
    build, libqsa_debug.so); returns the path that served them before."""
    global _lib, _lib_path
    prev = _lib_path
    _lib = _open(path)
    _lib_path = path
    return prev


def _open(path: str):
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m block_sparse_long_qsa_b200._build` "
                          "(the QSA path has no non-CUDA fallback)")
    L = ctypes.CDLL(path)
    P, vp, i64, i32, sz = ctypes.POINTER(qsa_params), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    psz = ctypes.POINTER(ctypes.c_size_t)
    L.qsa_default_params.argtypes = [P]
    L.qsa_default_params.restype = None
    L.qsa_status_string.argtypes = [ctypes.c_int]
    L.qsa_status_string.restype = ctypes.c_char_p
    L.qsa_last_error.argtypes = []
    L.qsa_last_error.restype = ctypes.c_char_p
    L.qsa_index_scores.argtypes = [P, i64, vp, vp, vp, i64, i64, vp, i64, vp, sz, vp]
    L.qsa_select_blocks.argtypes = [P, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.qsa_select_workspace_size.argtypes = [P, psz]
    L.qsa_index_workspace_size.argtypes = [P, i64, psz]
    L.qsa_prefill.argtypes = [P, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qsa_prefill_workspace_size.argtypes = [P, i64, psz, psz]
    L.qsa_prefill_cached.argtypes = [P, i64, i64] + [vp] * 16 + [sz, vp]
    L.qsa_prefill_cached_workspace_size.argtypes = [P, i64, i64, psz, psz]
    L.qsa_decode.argtypes = [P, i32, i64, ctypes.POINTER(ctypes.c_int64), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                             vp, vp, vp, vp, sz, vp]
    L.qsa_decode_workspace_size.argtypes = [P, i32, i64, psz]
    L.qsa_decode_mean_pool.argtypes = [P, i32, i64, ctypes.POINTER(ctypes.c_int64)] + [vp] * 15 + [vp, sz, vp]
    L.qsa_mean_pool_keys.argtypes = [P, i64, vp, vp, vp]
    L.qsa_verify.argtypes = [P, i32, i32, i64, ctypes.POINTER(ctypes.c_int64)] + [vp] * 15 + [vp, sz, vp]
    L.qsa_verify_workspace_size.argtypes = [P, i32, i32, i64, psz]
    L.qsa_decode_reuse.argtypes = [P, i32, i64, ctypes.POINTER(ctypes.c_int64)] + [vp] * 16 + [vp, sz, vp]
    L.qsa_decode_noalloc.argtypes = [P, i32, i64, ctypes.POINTER(ctypes.c_int64), vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp, vp, vp, vp, vp, vp, vp]
    L.qsa_check_device_error.argtypes = [vp, vp]
    L.qsa_decode_noalloc_check_error.argtypes = [vp]
    L.qsa_set_decode_splits.argtypes = [i32]
    LP, KV = ctypes.POINTER(qsa_layer_params), ctypes.POINTER(qsa_paged_kv)
    L.qsa_default_layer_params.argtypes = [LP]
    L.qsa_default_layer_params.restype = None
    L.qsa_norm_rope.argtypes = [LP, i64, i64, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp]
    L.qsa_paged_append.argtypes = [LP, KV, i32, i64, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, sz, vp]
    L.qsa_paged_decode.argtypes = [LP, KV, i32, vp, vp, vp, vp, vp, sz, vp]
    L.qsa_paged_prefill.argtypes = [LP, KV, i32, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qsa_paged_workspace_size.argtypes = [LP, i32, i64, psz]
    L.qsa_trace_begin.argtypes = [i32]
    L.qsa_trace_end.argtypes = [vp, vp, i32, ctypes.POINTER(ctypes.c_int32)]
    for f in EXPORTED:
        if f not in ("qsa_default_params", "qsa_default_layer_params", "qsa_status_string", "qsa_last_error"):
            getattr(L, f).restype = ctypes.c_int
    if hasattr(L, "qsa_debug_inject"):        # the debug build only
        L.qsa_debug_inject.argtypes = [i32]
        L.qsa_debug_inject.restype = ctypes.c_int
    _libs[path] = L
    return L


def params(budget: int = 512, **kw) -> qsa_params:
    p = qsa_params()
    load().qsa_default_params(ctypes.byref(p))
    p.budget_blocks = budget
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("QSA tensors must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, where: str):
    if rc != QSA_OK:
        detail = load().qsa_last_error().decode(errors="replace") if rc in (5, 8) else ""
        raise QSAError(rc, where, detail)


# ------------------------------------------------------------ raw entry points
def qsa_status_string(status: int) -> str:
    return load().qsa_status_string(status).decode()


def qsa_index_workspace_size(p: qsa_params, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load().qsa_index_workspace_size(ctypes.byref(p), T, ctypes.byref(n)), "qsa_index_workspace_size")
    return n.value


def qsa_index_scores(p: qsa_params, T: int, q_idx, w, k_idx, qb_begin: int, qb_end: int, scores, ld: int,
                     ws=None, stream=None):
    _check(load().qsa_index_scores(ctypes.byref(p), T, _ptr(q_idx), _ptr(w), _ptr(k_idx), qb_begin, qb_end,
                                   _ptr(scores), ld, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                   _stream(stream)), "qsa_index_scores")


def qsa_select_workspace_size(p: qsa_params) -> int:
    n = ctypes.c_size_t()
    _check(load().qsa_select_workspace_size(ctypes.byref(p), ctypes.byref(n)), "qsa_select_workspace_size")
    return n.value


def qsa_select_blocks(p: qsa_params, scores, ld: int, qb_begin: int, qb_end: int, sel, cnt, ws, stream=None):
    _check(load().qsa_select_blocks(ctypes.byref(p), _ptr(scores), ld, qb_begin, qb_end, _ptr(sel), _ptr(cnt),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "qsa_select_blocks")


def qsa_prefill_workspace_size(p: qsa_params, T: int) -> tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qsa_prefill_workspace_size(ctypes.byref(p), T, ctypes.byref(a), ctypes.byref(b)),
           "qsa_prefill_workspace_size")
    return a.value, b.value


def qsa_prefill(p: qsa_params, T: int, pos0: int, q, k, v, q_idx, w, k_idx, out, lse=None, sel_out=None,
                cnt_out=None, k_rot_out=None, ws=None, stream=None):
    _check(load().qsa_prefill(ctypes.byref(p), T, pos0, _ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(w), _ptr(k_idx),
                              _ptr(out), _ptr(lse), _ptr(sel_out), _ptr(cnt_out), _ptr(k_rot_out), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "qsa_prefill")


def qsa_prefill_cached_workspace_size(p: qsa_params, L_old: int, T_new: int) -> tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qsa_prefill_cached_workspace_size(ctypes.byref(p), L_old, T_new, ctypes.byref(a), ctypes.byref(b)),
           "qsa_prefill_cached_workspace_size")
    return a.value, b.value


def qsa_prefill_cached(p: qsa_params, L_old: int, T_new: int, k_cache, v_cache, kidx_cache, qidx_prev, w_prev, q, k,
                       v, q_idx, w, k_idx, out, lse=None, sel_out=None, cnt_out=None, ws=None, stream=None):
    _check(load().qsa_prefill_cached(ctypes.byref(p), L_old, T_new, _ptr(k_cache), _ptr(v_cache), _ptr(kidx_cache),
                                     _ptr(qidx_prev), _ptr(w_prev), _ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(w),
                                     _ptr(k_idx), _ptr(out), _ptr(lse), _ptr(sel_out), _ptr(cnt_out), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "qsa_prefill_cached")


def qsa_decode_workspace_size(p: qsa_params, B: int, max_len: int) -> int:
    n = ctypes.c_size_t()
    _check(load().qsa_decode_workspace_size(ctypes.byref(p), B, max_len, ctypes.byref(n)), "qsa_decode_workspace_size")
    return n.value


def qsa_decode(p: qsa_params, B: int, max_len: int, cache_len, k_cache, v_cache, kidx_cache, qidx_ring, w_ring,
               q_new, k_new, v_new, q_idx_new, k_idx_new, w_new, out, sel_out=None, lse_out=None, ws=None,
               stream=None):
    """``cache_len``: host sequence of B ints (lengths before this token)."""
    lens = (ctypes.c_int64 * B)(*[int(x) for x in cache_len])
    _check(load().qsa_decode(ctypes.byref(p), B, max_len, lens, _ptr(k_cache), _ptr(v_cache), _ptr(kidx_cache),
                             _ptr(qidx_ring), _ptr(w_ring), _ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(q_idx_new),
                             _ptr(k_idx_new), _ptr(w_new), _ptr(out), _ptr(sel_out), _ptr(lse_out), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "qsa_decode")


def qsa_decode_mean_pool(p: qsa_params, B: int, max_len: int, cache_len, k_cache, v_cache, kidx_cache, kbar_cache,
                         qidx_ring, w_ring, q_new, k_new, v_new, q_idx_new, k_idx_new, w_new, out, sel_out=None,
                         lse_out=None, ws=None, stream=None):
    lens = (ctypes.c_int64 * B)(*[int(x) for x in cache_len])
    _check(load().qsa_decode_mean_pool(ctypes.byref(p), B, max_len, lens, _ptr(k_cache), _ptr(v_cache),
                                       _ptr(kidx_cache), _ptr(kbar_cache), _ptr(qidx_ring), _ptr(w_ring),
                                       _ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(q_idx_new), _ptr(k_idx_new),
                                       _ptr(w_new), _ptr(out), _ptr(sel_out), _ptr(lse_out), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream)), "qsa_decode_mean_pool")


def qsa_decode_reuse(p: qsa_params, B: int, max_len: int, cache_len, k_cache, v_cache, kidx_cache, kbar_cache,
                     qidx_ring, w_ring, q_new, k_new, v_new, q_idx_new, k_idx_new, w_new, sel_in, cnt_in, out,
                     lse_out=None, ws=None, stream=None):
    """Draft decode step over a reused selection (``kbar_cache`` None unless
    the parameters select mean pooling)."""
    lens = (ctypes.c_int64 * B)(*[int(x) for x in cache_len])
    _check(load().qsa_decode_reuse(ctypes.byref(p), B, max_len, lens, _ptr(k_cache), _ptr(v_cache), _ptr(kidx_cache),
                                   _ptr(kbar_cache), _ptr(qidx_ring), _ptr(w_ring), _ptr(q_new), _ptr(k_new),
                                   _ptr(v_new), _ptr(q_idx_new), _ptr(k_idx_new), _ptr(w_new), _ptr(sel_in),
                                   _ptr(cnt_in), _ptr(out), _ptr(lse_out), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "qsa_decode_reuse")


def qsa_verify_workspace_size(p: qsa_params, B: int, m: int, max_len: int) -> int:
    n = ctypes.c_size_t()
    _check(load().qsa_verify_workspace_size(ctypes.byref(p), B, m, max_len, ctypes.byref(n)),
           "qsa_verify_workspace_size")
    return n.value


def qsa_verify(p: qsa_params, B: int, m: int, max_len: int, cache_len, k_cache, v_cache, kidx_cache, qidx_prev,
               w_prev, q_new, k_new, v_new, q_idx_new, k_idx_new, w_new, out, sel_out=None, lse_out=None, ws=None,
               stream=None, kbar_cache=None):
    """Verify m new tokens per sequence (``cache_len``: host sequence of B
    ints; ``kbar_cache`` only with mean-pooled parameters)."""
    lens = (ctypes.c_int64 * B)(*[int(x) for x in cache_len])
    _check(load().qsa_verify(ctypes.byref(p), B, m, max_len, lens, _ptr(k_cache), _ptr(v_cache), _ptr(kidx_cache),
                             _ptr(kbar_cache), _ptr(qidx_prev), _ptr(w_prev), _ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(q_idx_new),
                             _ptr(k_idx_new), _ptr(w_new), _ptr(out), _ptr(sel_out), _ptr(lse_out), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "qsa_verify")


def qsa_mean_pool_keys(p: qsa_params, T: int, k_idx, kbar, stream=None):
    _check(load().qsa_mean_pool_keys(ctypes.byref(p), T, _ptr(k_idx), _ptr(kbar), _stream(stream)),
           "qsa_mean_pool_keys")


def qsa_decode_noalloc(p: qsa_params, B: int, max_len: int, cache_len, k_cache, v_cache, kidx_cache, qidx_ring,
                       w_ring, q_new, k_new, v_new, q_idx_new, k_idx_new, w_new, out, sel_out=None, lse_out=None,
                       stream=None):
    """qsa_decode on the library's fixed scratch array (no workspace, no allocation)."""
    lens = (ctypes.c_int64 * B)(*[int(x) for x in cache_len])
    _check(load().qsa_decode_noalloc(ctypes.byref(p), B, max_len, lens, _ptr(k_cache), _ptr(v_cache),
                                     _ptr(kidx_cache), _ptr(qidx_ring), _ptr(w_ring), _ptr(q_new), _ptr(k_new),
                                     _ptr(v_new), _ptr(q_idx_new), _ptr(k_idx_new), _ptr(w_new), _ptr(out),
                                     _ptr(sel_out), _ptr(lse_out), _stream(stream)), "qsa_decode_noalloc")


# ------------------------------------------------- layers over a paged cache
def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# torch's own C entries where it has them: the public functions wrap them in
# Python (about 2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_ELEMENT = (torch.bfloat16, torch.float16)     # by qsa_layer_params.dtype


def layer_params(n_q_heads: int = 24, n_kv_heads: int = 2, head_dim: int = 256, dtype=torch.bfloat16,
                 rope_section=None, **kw) -> qsa_layer_params:
    """qsa_layer_params with its defaults; ``dtype``: torch.bfloat16 or
    torch.float16, ``rope_section``: rotary pairs of time, height, width."""
    p = qsa_layer_params()
    load().qsa_default_layer_params(ctypes.byref(p))
    p.n_q_heads, p.n_kv_heads, p.head_dim = n_q_heads, n_kv_heads, head_dim
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("dtype must be torch.bfloat16 or torch.float16")
    p.dtype = DTYPE_FP16 if dtype == torch.float16 else DTYPE_BF16
    if rope_section is not None:
        p.rope_section[:] = [int(x) for x in rope_section]
    for k, v in kw.items():
        if k not in _LAYER_FIELDS:
            raise TypeError(f"qsa_layer_params has no field {k}")
        setattr(p, k, v)
    return p


_LAYER_FIELDS = {n for n, _ in qsa_layer_params._fields_}


class PagedKV:
    """A paged cache of the paged calls: ``k_pages`` and ``v_pages``
    [n_pages][page_size][n_kv_heads][head_dim] (any strides of whole 16-byte
    units, alike for both; head-major pools pass ``pool.transpose(1, 2)``) and
    ``page_table`` [B][max_pages] int32, all on one device.  Holds references to
    the three tensors; ``c`` is the C struct."""

    def __init__(self, k_pages, v_pages, page_table):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride():
            raise ValueError("k_pages and v_pages must be alike, [n_pages][page_size][n_kv_heads][head_dim]")
        if k_pages.dtype != v_pages.dtype or k_pages.element_size() != 2:
            raise ValueError("k_pages and v_pages must have one 16-bit dtype")
        if k_pages.shape[3] > 1 and k_pages.stride(3) != 1:
            raise ValueError("a page row's elements must be contiguous")
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be int32 [B][max_pages] with contiguous rows")
        if not (k_pages.device == v_pages.device == page_table.device):
            raise ValueError("k_pages, v_pages and page_table must be on one device")
        if 0 in k_pages.shape or page_table.shape[1] == 0:
            raise ValueError("k_pages and page_table must not be empty")
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        # the stride of a dimension of one entry is never used
        d = k_pages.shape[3]
        st = [s if n > 1 else max(d, s) // 8 * 8 for n, s in zip(k_pages.shape, k_pages.stride())]
        ld = page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1]
        self.heads, self.dtype = tuple(k_pages.shape[2:]), k_pages.dtype
        self.rows, self.device = page_table.shape[0], k_pages.get_device()
        self.c = qsa_paged_kv(k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[0], k_pages.shape[1],
                              page_table.shape[1], st[0], st[1], st[2], page_table.data_ptr(), ld)
        self.ref = ctypes.byref(self.c)


def _flat(t, what: str, shape, dt, dev: int):
    """Pointer of a contiguous tensor of the given shape (rows may be more),
    dtype (``dt``, or bit patterns in torch.uint16 for a 16-bit one) and device
    index; None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dt or t.get_device() != dev or not t.is_contiguous():
        if t.dim() != len(shape) or t.shape[0] < shape[0] or tuple(t.shape[1:]) != shape[1:]:
            raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
        if t.dtype is not dt and not (t.dtype is torch.uint16 and dt in _ELEMENT):
            raise ValueError(f"{what} has dtype {t.dtype}, not {dt}")
        if t.get_device() != dev:
            raise ValueError(f"{what} is on {t.device}, not on the device of the other tensors")
        if not t.is_contiguous():
            raise ValueError("QSA tensors must be contiguous")
    return t.data_ptr()


def _rows(t, what: str, T: int, H: int, D: int, dt, dev: int):
    """(pointer, row stride) of a [T][H][D] tensor whose rows are contiguous inside."""
    if t is None:
        return None, 0
    st = t.stride()
    if t.shape != (T, H, D) or t.dtype is not dt or t.get_device() != dev or st[2] != 1 or st[1] != D or T < 2:
        if t.dim() != 3 or t.shape[0] < T or t.shape[1] != H or t.shape[2] != D:
            raise ValueError(f"{what} must be [{T}][{H}][{D}], not {list(t.shape)}")
        if t.dtype is not dt and t.dtype is not torch.uint16:
            raise ValueError(f"{what} has dtype {t.dtype}, the layer {dt}")
        if t.get_device() != dev:
            raise ValueError(f"{what} is on {t.device}, not on the device of the other tensors")
        if st[2] != 1 or (H > 1 and st[1] != D):
            raise ValueError(f"the heads of a row of {what} must be contiguous")
        if t.shape[0] < 2:
            return t.data_ptr(), H * D          # the stride of a single row is never used
    return t.data_ptr(), st[0]


def _positions(positions, axes: int, T: int, dev: int):
    if positions is None:
        return None
    if axes == 1 and positions.dim() == 1:
        positions = positions[None]
    if positions.shape != (axes, T):
        raise ValueError(f"positions must be [{axes}][{T}], not {list(positions.shape)}")
    return _flat(positions, "positions", (axes, T), torch.int32, dev)


def _paged(p, kv: "PagedKV", B: int, ws):
    """Checks of the cache against the layer; (device index, element type, workspace pointer and bytes)."""
    dt = _ELEMENT[p.dtype]
    if kv.heads != (p.n_kv_heads, p.head_dim):
        raise ValueError(f"the pages hold {list(kv.heads)}, the layer [{p.n_kv_heads}, {p.head_dim}]")
    if kv.dtype is not dt and kv.dtype is not torch.uint16:
        raise ValueError(f"the pages have dtype {kv.dtype}, the layer {dt}")
    if kv.rows < B:
        raise ValueError(f"page_table has {kv.rows} rows for {B} sequences")
    if ws is None or ws.get_device() != kv.device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous workspace on the cache's device (paged_workspace)")
    return kv.device, dt, ws.data_ptr(), ws.numel() * ws.element_size()


def _run(fn: str, dev: int, stream, *args):
    """The C call ``fn`` with ``dev`` current, on ``stream`` or on that device's current stream."""
    if dev < 0:
        raise ValueError(f"{fn}: the tensors are not on a CUDA device")
    f = getattr(_lib or load(), fn)
    s = stream.cuda_stream if stream is not None else _raw_stream(dev)
    if dev == _current_device():
        rc = f(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, s)
    if rc != QSA_OK:
        _check(rc, fn)


def qsa_norm_rope(p: qsa_layer_params, T: int, pos0: int, q, k, q_weight, k_weight, q_out, k_out, positions=None,
                  stream=None):
    """``q`` [T][n_q_heads][head_dim], ``k`` [T][n_kv_heads][head_dim] (row
    strides free); ``q`` with ``q_out``, or ``k`` with ``k_out``, and each weight
    may be None; ``positions`` int32 [rope_axes][T]."""
    if q is None and k is None:
        raise ValueError("one of q and k is needed")
    dev, dt = (q if q is not None else k).get_device(), _ELEMENT[p.dtype]
    H, G, D = p.n_q_heads, p.n_kv_heads, p.head_dim
    qp, ql = _rows(q, "q", T, H, D, dt, dev)
    kp, kl = _rows(k, "k", T, G, D, dt, dev)
    _run("qsa_norm_rope", dev, stream, ctypes.byref(p), T, pos0, _positions(positions, p.rope_axes, T, dev), qp, ql, kp,
         kl, _flat(q_weight, "q_weight", (D,), dt, dev), _flat(k_weight, "k_weight", (D,), dt, dev),
         _flat(q_out, "q_out", (T, H, D), dt, dev), _flat(k_out, "k_out", (T, G, D), dt, dev))


def qsa_paged_append(p: qsa_layer_params, kv: PagedKV, B: int, T: int, cu_new, cache_len, k, v, ws, q=None, q_out=None,
                     q_weight=None, k_weight=None, positions=None, stream=None):
    """``cu_new`` int32 [B + 1] or None (one token per sequence), ``cache_len``
    int32 [B], both on the device."""
    dev, dt, wp, wb = _paged(p, kv, B, ws)
    H, G, D = p.n_q_heads, p.n_kv_heads, p.head_dim
    qp, ql = _rows(q, "q", T, H, D, dt, dev)
    kp, kl = _rows(k, "k", T, G, D, dt, dev)
    vp, vl = _rows(v, "v", T, G, D, dt, dev)
    _run("qsa_paged_append", dev, stream, ctypes.byref(p), kv.ref, B, T,
         _flat(cu_new, "cu_new", (B + 1,), torch.int32, dev), _flat(cache_len, "cache_len", (B,), torch.int32, dev),
         _positions(positions, p.rope_axes, T, dev), qp, ql, kp, kl, vp, vl,
         _flat(q_weight, "q_weight", (D,), dt, dev), _flat(k_weight, "k_weight", (D,), dt, dev),
         _flat(q_out, "q_out", (T, H, D), dt, dev), wp, wb)


def qsa_paged_decode(p: qsa_layer_params, kv: PagedKV, B: int, cache_len, q, out, ws, lse=None, stream=None):
    """One new token per sequence (``q``, ``out`` [B][n_q_heads][head_dim])."""
    dev, dt, wp, wb = _paged(p, kv, B, ws)
    H, D = p.n_q_heads, p.head_dim
    _run("qsa_paged_decode", dev, stream, ctypes.byref(p), kv.ref, B,
         _flat(cache_len, "cache_len", (B,), torch.int32, dev), _flat(q, "q", (B, H, D), dt, dev),
         _flat(out, "out", (B, H, D), dt, dev), _flat(lse, "lse", (B, H), torch.float32, dev), wp, wb)


def qsa_paged_prefill(p: qsa_layer_params, kv: PagedKV, B: int, T: int, cu_new, cache_len, q, out, ws, lse=None,
                      stream=None):
    """T new tokens of B sequences (``q``, ``out`` [T][n_q_heads][head_dim])."""
    dev, dt, wp, wb = _paged(p, kv, B, ws)
    H, D = p.n_q_heads, p.head_dim
    _run("qsa_paged_prefill", dev, stream, ctypes.byref(p), kv.ref, B, T,
         _flat(cu_new, "cu_new", (B + 1,), torch.int32, dev), _flat(cache_len, "cache_len", (B,), torch.int32, dev),
         _flat(q, "q", (T, H, D), dt, dev), _flat(out, "out", (T, H, D), dt, dev),
         _flat(lse, "lse", (T, H), torch.float32, dev), wp, wb)


def qsa_paged_workspace_size(p: qsa_layer_params, B: int, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load().qsa_paged_workspace_size(ctypes.byref(p), B, T, ctypes.byref(n)), "qsa_paged_workspace_size")
    return n.value


def paged_workspace(p: qsa_layer_params, B: int, T: int, device="cuda") -> torch.Tensor:
    """A workspace of the paged calls with its error word cleared."""
    ws = torch.empty(qsa_paged_workspace_size(p, B, T), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def qsa_check_device_error(ws, stream=None) -> int:
    return load().qsa_check_device_error(_ptr(ws), _stream(stream))


def qsa_decode_noalloc_check_error(stream=None) -> int:
    """Device error word of qsa_decode_noalloc's fixed array (synchronises)."""
    return load().qsa_decode_noalloc_check_error(_stream(stream))


# fault-injection codes of the debug build (include/qsa_debug.h)
INJECT_INDEXER_STALL = 1
INJECT_ATTENTION_STALL = 2
INJECT_ATTENTION_BAD_BLOCK = 3
INJECT_ATTENTION_RESCALE_ALL = 4
INJECT_PAGED_STALL = 5


def qsa_debug_inject(code: int):
    """Arm a test fault for the next launch of the kernel it names (the debug
    build, libqsa_debug.so, only)."""
    L = load()
    if not hasattr(L, "qsa_debug_inject"):
        raise RuntimeError("qsa_debug_inject exists only in the debug build (use_library(LIB_DEBUG_PATH))")
    _check(L.qsa_debug_inject(int(code)), "qsa_debug_inject")


def qsa_set_decode_splits(n: int):
    """Fix the number of split-KV decode ranges (1..16) for this process; 0 = automatic."""
    _check(load().qsa_set_decode_splits(int(n)), "qsa_set_decode_splits")


class trace:
    """Context manager: per-launch device times of this library's kernels,
    from CUDA events recorded on each launching stream.  ``.records`` is a
    list of (kernel name, milliseconds) in launch order."""

    def __init__(self, capacity: int = 4096):
        self.capacity = capacity
        self.records = []

    def __enter__(self):
        _check(load().qsa_trace_begin(self.capacity), "qsa_trace_begin")
        return self

    def __exit__(self, *exc):
        ids = (ctypes.c_int32 * self.capacity)()
        ms = (ctypes.c_float * self.capacity)()
        n = ctypes.c_int32()
        _check(load().qsa_trace_end(ids, ms, self.capacity, ctypes.byref(n)), "qsa_trace_end")
        self.records = [(KERNEL_NAMES.get(ids[i], str(ids[i])), ms[i]) for i in range(n.value)]
        return False

    def by_kernel(self) -> dict:
        out = {}
        for name, t in self.records:
            c, tot = out.get(name, (0, 0.0))
            out[name] = (c + 1, tot + t)
        return out


# ----------------------------------------------------- allocating conveniences
def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def prefill(q, k, v, q_idx, w, k_idx, budget: int = 512, pos0: int = 0, want_lse=True, want_sel=True,
            want_krot=False, ws_bytes: int | None = None, stream=None, aggregation: int = AGG_TOKEN_MAX,
            idx_rope: int = 0):
    """Allocate outputs and a workspace, run qsa_prefill; returns a dict."""
    T = q.shape[0]
    dev = q.device
    p = params(budget, aggregation=aggregation, idx_rope=idx_rope)
    mn, pref = qsa_prefill_workspace_size(p, T)
    ws = workspace(pref if ws_bytes is None else max(ws_bytes, mn), dev)
    nqb = (T + 3) // 4
    res = dict(out=torch.empty((T, 24, 256), dtype=torch.uint16, device=dev))
    res["lse"] = torch.empty((T, 24), dtype=torch.float32, device=dev) if want_lse else None
    res["sel"] = torch.empty((nqb, budget), dtype=torch.int32, device=dev) if want_sel else None
    res["cnt"] = torch.empty((nqb,), dtype=torch.int32, device=dev) if want_sel else None
    res["k_rot"] = torch.empty((T, 2, 256), dtype=torch.uint16, device=dev) if want_krot else None
    qsa_prefill(p, T, pos0, q, k, v, q_idx, w, k_idx, res["out"], res["lse"], res["sel"], res["cnt"], res["k_rot"],
                ws, stream)
    res["ws"] = ws
    return res
