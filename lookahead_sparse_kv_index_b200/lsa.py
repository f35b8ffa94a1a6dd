"""Thin ctypes binding of liblsa.so (include/lsa.h).

Argument marshalling only: torch tensors supply device memory and streams,
every step of the path runs in the library's CUDA kernels.  There is no CPU
fallback: if liblsa.so is missing or cannot be loaded, importing this module
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblsa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m lookahead_sparse_kv_index_b200.build`")
_L = ctypes.CDLL(LIB_PATH)

P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

F32, BF16, E4M3 = 0, 1, 2
DTYPE = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
STATUS = {0: "LSA_OK", 1: "LSA_ERR_INVALID", 2: "LSA_ERR_CUDA", 3: "LSA_ERR_CAPACITY", 4: "LSA_ERR_TIMEOUT",
          5: "LSA_ERR_UNSUPPORTED"}
(STAGE_SCORE, STAGE_SELECT, STAGE_GATHER, STAGE_TOPK, STAGE_ATTN, STAGE_RESCORE) = range(6)
STAGES = ["score", "select", "gather", "topk", "attn", "rescore"]
N_STAGES = 6

# every symbol include/lsa.h declares
EXPORTS = [
    "lsa_version", "lsa_last_error", "lsa_last_kernel", "lsa_status_name", "lsa_index_score",
    "lsa_select_workspace_size", "lsa_select_noalloc_max_entries", "lsa_select_noalloc",
    "lsa_select", "lsa_topk", "lsa_gather", "lsa_sparse_attn_workspace_size", "lsa_sparse_attn",
    "lsa_ctx_create", "lsa_ctx_destroy", "lsa_decode_step", "lsa_decode_step_host", "lsa_ctx_get_view",
    "lsa_ctx_set_graphs", "lsa_ctx_set_timing", "lsa_ctx_stage_times", "lsa_ctx_reset_counters",
    "lsa_ctx_launches", "lsa_selftest_bounded_wait", "lsa_index_union", "lsa_query_encode",
    "lsa_attn_set_merge", "lsa_struct_size", "lsa_ctx_flush_cache", "lsa_index_score_select_workspace_size",
    "lsa_index_score_select", "lsa_paged_attn_workspace_size", "lsa_paged_attn", "lsa_qk_norm_rope",
    "lsa_rope_frequencies", "lsa_page_grow", "lsa_page_fork", "lsa_page_free", "lsa_page_compact_workspace_size",
    "lsa_page_compact", "lsa_page_copy",
]


class LsaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _L.lsa_last_error().decode()
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")


class Params(ctypes.Structure):
    _fields_ = [
        ("B", i32), ("H", i32), ("d", i32), ("q_dtype", i32), ("k_dtype", i32),
        ("Hq", i32), ("D", i32), ("attn_dtype", i32), ("topk", i32), ("tau", i32), ("scale", f32),
        ("n_total", i64), ("seq_off_host", P), ("k_dev", P), ("k_scale_dev", P), ("cold_host", P),
        ("row_bytes", i64), ("kv_row_stride", i64), ("k_off", i64), ("v_off", i64), ("kept_capacity", i64),
        ("full_fetch", i32), ("window", i32), ("hca_rows", P), ("hca_off_host", P),
        ("n_layers", i32), ("k_dev_layers", P), ("k_scale_layers", P), ("lookahead", i32),
    ]


class View(ctypes.Structure):
    _fields_ = [("z", P), ("z_kept", P), ("kept_idx", P), ("kept_off", P), ("slot_of", P), ("hot", P),
                ("topk_idx", P), ("topk_pos", P), ("topk_cnt", P), ("err", P), ("kept_slot", P), ("owner", P),
                ("fetched", P), ("attn_rows", P), ("attn_row_cap", i64), ("win_base", i64), ("hca_base", i64)]


class PageCacheDesc(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("dtype", i32), ("page_size", i32), ("Hkv", i32),
                ("D", i32), ("n_pages", i64), ("page_stride", i64), ("slot_stride", i64), ("head_stride", i64)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("freq", P), ("rot_dim", i32), ("interleaved", i32), ("inverse", i32), ("mscale", f32)]


class PageTableDesc(ctypes.Structure):
    _fields_ = [("table", P), ("len", P), ("refs", P), ("n_rows", i32), ("max_pages", i32), ("page_size", i32),
                ("n_pages", i64)]


def _sig(name, res, args):
    f = getattr(_L, name)
    f.restype = res
    f.argtypes = args


_sig("lsa_version", i32, [])
_sig("lsa_struct_size", i64, [i32])
_sig("lsa_last_error", ctypes.c_char_p, [])
_sig("lsa_last_kernel", ctypes.c_char_p, [])
_sig("lsa_status_name", ctypes.c_char_p, [i32])
_sig("lsa_index_score", i32, [P, i32, P, P, i32, P, P, i64, P, P, i64, i32, i32, i32, P, P, i32, P, P])
SCORE_CUDA_CORE = 1
_sig("lsa_select_workspace_size", sz, [i64])
_sig("lsa_index_score_select_workspace_size", sz, [i64, i32])
_sig("lsa_index_score_select", i32, [P, i32, P, P, i32, P, P, i64, i32, i32, i32, P, P, i64, P, P, sz, P, P])
_sig("lsa_select", i32, [P, P, i64, i32, P, i64, P, P, P, sz, P, P])
_sig("lsa_select_noalloc_max_entries", i64, [])
_sig("lsa_select_noalloc", i32, [P, P, i64, i32, P, i64, P, P, P, P])
_sig("lsa_topk", i32, [P, i32, P, P, P, i64, i32, i32, P, P, P, P])
_sig("lsa_gather", i32, [P, i64, P, i64, P, P, i32, P, i64, P, P, P])
_sig("lsa_sparse_attn_workspace_size", sz, [i32, i32, i32, i32])
_sig("lsa_sparse_attn", i32, [P, i32, P, i64, i64, i64, P, i32, i32, i32, i32, f32, P, P, P, sz, P, P])
_sig("lsa_ctx_create", i32, [ctypes.POINTER(Params), ctypes.POINTER(P)])
_sig("lsa_ctx_destroy", i32, [P])
_sig("lsa_decode_step", i32, [P, i64, P, P, P, P, P, P])
_sig("lsa_decode_step_host", i32, [P, i64, P, P, P, P, P, P])
_sig("lsa_ctx_get_view", i32, [P, ctypes.POINTER(View)])
_sig("lsa_ctx_set_graphs", i32, [P, i32])
_sig("lsa_ctx_set_timing", i32, [P, i32])
_sig("lsa_ctx_stage_times", i32, [P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)])
_sig("lsa_ctx_reset_counters", i32, [P])
_sig("lsa_ctx_launches", i64, [P])
_sig("lsa_ctx_flush_cache", i32, [P, P])
_sig("lsa_selftest_bounded_wait", i32, [i64, P, P, P])
_sig("lsa_index_union", i32, [ctypes.POINTER(P), i32, i64, P, P])
_sig("lsa_query_encode", i32, [P, i32, i32, P, i32, P, i32, i32, P, P, i32, P, P, P])
_sig("lsa_attn_set_merge", i32, [P, P, P, P, i32, i32, i32, i32, P, i32, P, i32, P, P, P])
_sig("lsa_paged_attn_workspace_size", sz, [P, i32, i32])
_sig("lsa_paged_attn", i32, [P, i32, i64, P, P, i64, i32, P, i32, i32, i32, f32, P, P, P, sz, P, P])
_sig("lsa_qk_norm_rope", i32, [P, i64, P, i64, P, i64, P, i64, P, i64, i32, i64, i32, i32, i32, P, P, f32, P, P, P, P,
                               i64, i32, i32, P, P, P, P])
_sig("lsa_rope_frequencies", i32, [i32, i32, ctypes.c_double, ctypes.c_double, i64, ctypes.c_double, ctypes.c_double,
                                   P, P])
_sig("lsa_page_grow", i32, [P, P, P, P])
_sig("lsa_page_fork", i32, [P, P, P, i32, P, P, P, P])
_sig("lsa_page_free", i32, [P, P, i32, P, P])
_sig("lsa_page_compact_workspace_size", sz, [i64])
_sig("lsa_page_compact", i32, [P, P, P, P, P, P, P, sz, P])
_sig("lsa_page_copy", i32, [P, P, P, i32, P, P, P])

lib = _L


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(status, where):
    if status != 0:
        raise LsaError(status, where)


def version() -> int:
    return int(_L.lsa_version())


def last_kernel() -> str:
    """Name of the last kernel this thread launched through the library."""
    return _L.lsa_last_kernel().decode()


# ------------------------------------------------------------------ stages

def index_score(q, q_dtype, w, k, k_dtype, k_scale, seq_off, n_total, H, d, z, I=None, idx=None, idx_off=None,
                list_capacity=0, cuda_core=False, err=None, stream=None):
    """Lookahead index score; cuda_core=True forces the CUDA-core kernel (else tcgen05 where supported)."""
    B = seq_off.numel() - 1
    _check(_L.lsa_index_score(_ptr(q), DTYPE[q_dtype], _ptr(w), _ptr(k), DTYPE[k_dtype], _ptr(k_scale),
                              _ptr(seq_off), n_total, _ptr(idx), _ptr(idx_off), list_capacity, B, H, d,
                              _ptr(z), _ptr(I), SCORE_CUDA_CORE if cuda_core else 0, _ptr(err), _stream(stream)),
           "lsa_index_score")


def select_workspace_size(n_total) -> int:
    return int(_L.lsa_select_workspace_size(n_total))


def index_score_select_workspace_size(n_total, B) -> int:
    return int(_L.lsa_index_score_select_workspace_size(n_total, B))


def index_score_select(q, q_dtype, w, k, k_dtype, k_scale, seq_off, n_total, H, d, z, kept_idx, capacity, kept_off,
                       workspace, err=None, stream=None):
    """Full index scan and threshold selection in one call (fused on the tensor-core path; see lsa.h)."""
    B = seq_off.numel() - 1
    _check(_L.lsa_index_score_select(_ptr(q), DTYPE[q_dtype], _ptr(w), _ptr(k), DTYPE[k_dtype], _ptr(k_scale),
                                     _ptr(seq_off), n_total, B, H, d, _ptr(z), _ptr(kept_idx), capacity,
                                     _ptr(kept_off), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _ptr(err), _stream(stream)), "lsa_index_score_select")


def select(z, seq_off, n_total, kept_idx, capacity, kept_off, mask, workspace, err, stream=None):
    B = seq_off.numel() - 1
    _check(_L.lsa_select(_ptr(z), _ptr(seq_off), n_total, B, _ptr(kept_idx), capacity, _ptr(kept_off), _ptr(mask),
                         _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
                         _stream(stream)), "lsa_select")


def select_noalloc_max_entries() -> int:
    return int(_L.lsa_select_noalloc_max_entries())


def select_noalloc(z, seq_off, n_total, kept_idx, capacity, kept_off, mask, err, stream=None):
    """lsa_select with the library's static scratch instead of a caller workspace."""
    B = seq_off.numel() - 1
    _check(_L.lsa_select_noalloc(_ptr(z), _ptr(seq_off), n_total, B, _ptr(kept_idx), capacity, _ptr(kept_off),
                                 _ptr(mask), _ptr(err), _stream(stream)), "lsa_select_noalloc")


def index_union(z_layers, n_total, z_union, stream=None):
    """OR-mode union of indexer layers: z_union = max over the layers' scores (see lsa.h)."""
    arr = (P * len(z_layers))(*[_ptr(z) for z in z_layers])
    _check(_L.lsa_index_union(arr, len(z_layers), n_total, _ptr(z_union), _stream(stream)), "lsa_index_union")


def query_encode(h, W_dq, W_uq, W_w, H, d, q_out, q_dtype, w_out, c_out, stream=None):
    """Indexer query encoder: c = W_dq h, q = W_uq c as [B,H,d], w = W_w h (see lsa.h).  h: bf16 [B,hidden];
    W_dq [rank,hidden], W_uq [H*d,rank], W_w [H,hidden] bf16 (any 2-byte tensors holding bf16 bits)."""
    B, hidden = h.shape
    rank = W_dq.shape[0]
    _check(_L.lsa_query_encode(_ptr(h), B, hidden, _ptr(W_dq), rank, _ptr(W_uq), H, d, _ptr(W_w), _ptr(q_out),
                               DTYPE[q_dtype], _ptr(w_out), _ptr(c_out), _stream(stream)), "lsa_query_encode")


def attn_set_merge(topk_idx, topk_pos, topk_cnt, seq_off, k, window, win_base, hca_off, hca_base, rows, row_cap,
                   count=None, err=None, stream=None):
    """Merged attention set: per sequence the row list top-k (outside the window) + HCA rows + window rows."""
    B = seq_off.numel() - 1
    _check(_L.lsa_attn_set_merge(_ptr(topk_idx), _ptr(topk_pos), _ptr(topk_cnt), _ptr(seq_off), B, k, window,
                                 win_base, _ptr(hca_off), hca_base, _ptr(rows), row_cap, _ptr(count), _ptr(err),
                                 _stream(stream)), "lsa_attn_set_merge")


def selftest_bounded_wait(limit_ns, err, waited_ns, stream=None):
    """Runs a bounded device wait on a barrier nothing arrives at (see lsa.h)."""
    _check(_L.lsa_selftest_bounded_wait(int(limit_ns), _ptr(err), _ptr(waited_ns), _stream(stream)),
           "lsa_selftest_bounded_wait")


def topk(z, z_by_entry, seq_off, kept_idx, kept_off, kept_capacity, k, topk_idx, topk_pos, topk_cnt, stream=None):
    B = kept_off.numel() - 1
    _check(_L.lsa_topk(_ptr(z), int(z_by_entry), _ptr(seq_off), _ptr(kept_idx), _ptr(kept_off), kept_capacity, B, k,
                       _ptr(topk_idx), _ptr(topk_pos), _ptr(topk_cnt), _stream(stream)), "lsa_topk")


def gather(cold_host, row_bytes, seq_off, n_total, kept_idx, kept_off, hot, hot_capacity, slot_of, err,
           stream=None):
    B = seq_off.numel() - 1
    _check(_L.lsa_gather(_ptr(cold_host), row_bytes, _ptr(seq_off), n_total, _ptr(kept_idx), _ptr(kept_off), B,
                         _ptr(hot), hot_capacity, _ptr(slot_of), _ptr(err), _stream(stream)), "lsa_gather")


def sparse_attn_workspace_size(B, Hq, D, k) -> int:
    return int(_L.lsa_sparse_attn_workspace_size(B, Hq, D, k))


def sparse_attn(Q, dtype, kv, kv_row_stride, k_off, v_off, rows, B, Hq, D, k, scale, out, lse, workspace,
                err=None, stream=None):
    _check(_L.lsa_sparse_attn(_ptr(Q), DTYPE[dtype], _ptr(kv), kv_row_stride, k_off, v_off, _ptr(rows), B, Hq, D,
                              k, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)),
           "lsa_sparse_attn")


# -------------------------------------------------------------- paged cache
#
# These bindings read sizes, strides and types off the tensors, so they check them: a mismatch is a ValueError, and
# what the library refuses is an LsaError.  They run on the device that holds the tensors, on its current stream
# unless `stream` is given (a stream of that device).  A decode step calls them once a layer, where a call's host time
# is its cost: the checks build no message unless one fails, and the stream's handle is read without a Stream object.

_ELEM = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}
_I32, _FP32 = torch.int32, torch.float32


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _fits(x, name):
    """Refuses a number that an int32 argument would take modulo 2^32."""
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name}={x} is no int32")


def _i32(t, name, device, *shape):
    """The address of a contiguous int32 tensor of `shape` on `device`."""
    if t.dtype is not _I32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor {list(shape)} on {device} is needed, not {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def _err_word(err, device):
    if err is None:
        return None
    if err.dtype is not _I32 or err.device != device or err.numel() != 1:
        raise ValueError(f"err: one int32 on {device} is needed")
    return err.data_ptr()


def _room(t, device):
    """The address and bytes of a workspace."""
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on {device} is needed")
    return t.data_ptr(), t.numel() * t.element_size()


def _on(device, f, args, where, stream):
    """Calls the library with `device` current and its current stream, or the one given, as the last argument."""
    i = device.index
    if device.type != "cuda" or i is None:
        raise ValueError(f"{where}: tensors on a CUDA device are needed, not on {device}")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(i)
    elif stream.device == device:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"{where}: the stream is not one of {device}")
    if torch._C._cuda_getDevice() == i:
        status = f(*args, handle)
    else:
        with torch.cuda.device(device):
            status = f(*args, handle)
    if status:
        raise LsaError(status, where)


class PageCache:
    """One layer's paged key-value cache (lsa_page_cache in lsa.h).

    k, v: tensors [n_pages, page_size, Hkv, D] of float32, bfloat16 or float8_e4m3fn with the same strides, unit
    stride in D (a permuted view of another layout is fine); v None: a latent cache, whose rows are keys and values.
    k_scale, v_scale: contiguous float32 [n_pages, page_size, Hkv] for float8_e4m3fn rows.
    """

    def __init__(self, k, v=None, k_scale=None, v_scale=None):
        _need(k.dim() == 4 and k.dtype in _ELEM and k.stride(3) == 1,
              "k: [n_pages, page_size, Hkv, D] of float32, bfloat16 or float8_e4m3fn with unit stride in D is needed")
        _need(v is None or (v.shape == k.shape and v.stride() == k.stride() and v.dtype == k.dtype
                            and v.device == k.device), "v: the shape, strides, type and device of k are needed")
        _need(not (v is None and v_scale is not None), "v_scale goes with v")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(s is None or (s.dtype is _FP32 and s.shape == k.shape[:3] and s.is_contiguous()
                                and s.device == k.device),
                  f"{name}: a contiguous float32 tensor {list(k.shape[:3])} on {k.device} is needed")
        if v is None:
            v, v_scale = k, k_scale
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.n_pages, self.page_size, self.Hkv, self.D = k.shape
        self.desc = PageCacheDesc(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ELEM[k.dtype], self.page_size,
                                  self.Hkv, self.D, self.n_pages, k.stride(0), k.stride(1), k.stride(2))
        self._ref = ctypes.byref(self.desc)


def paged_attn_workspace_size(cache, B, Hq) -> int:
    """Bytes of paged_attn's workspace on the cache's device (raises on heads that the library does not run)."""
    _fits(B, "B")
    _fits(Hq, "Hq")
    if cache.device.type != "cuda" or cache.device.index == torch._C._cuda_getDevice():
        n = _L.lsa_paged_attn_workspace_size(cache._ref, B, Hq)
    else:
        with torch.cuda.device(cache.device):
            n = _L.lsa_paged_attn_workspace_size(cache._ref, B, Hq)
    _need(n > 0, _L.lsa_last_error().decode() or f"B={B} must be positive")
    return int(n)


def _table(t, device):
    """Address, row stride and shape of a page table."""
    if t.dtype is not _I32 or t.device != device or t.dim() != 2:
        raise ValueError(f"table: int32 [rows, max_pages] on {device} is needed, not {t.dtype} {list(t.shape)} on "
                         f"{t.device}")
    (rows, width), (step, unit) = t.shape, t.stride()
    if unit != 1 and width > 1:
        raise ValueError("table: unit stride along a row is needed")
    return t.data_ptr(), step if rows > 1 else width, rows, width


def _heads(t, name, T, H, D, dtype, device):
    """Address and token stride of heads [T, H, D] that lie side by side in a token."""
    step = t.stride()
    if (t.shape != (T, H, D) or t.dtype is not dtype or t.device != device or step[2] != 1
            or (step[1] != D and H > 1)):
        raise ValueError(f"{name}: [{T}, {H}, {D}] of {dtype} on {device} with heads side by side is needed, not "
                         f"{t.dtype} {list(t.shape)} with strides {list(step)} on {t.device}")
    return t.data_ptr(), step[0] if T > 1 else H * D


def paged_attn(Q, cache, table, seq_len, out, workspace, lse=None, window=0, scale=None, err=None, stream=None):
    """Attention of one new token per sequence over a PageCache (lsa_paged_attn).

    Q [B, Hq, D] (any stride between sequences), table int32 [B, max_pages], seq_len int32 [B]; out [B, Hq, D] and
    lse float32 [B, Hq] contiguous; workspace: a contiguous tensor of paged_attn_workspace_size bytes.  window: attend
    only the last `window` entries (0: all).  scale None: 1 / sqrt(D).
    """
    dev, dtype = cache.device, Q.dtype
    B, Hq, D = Q.shape
    _fits(window, "window")
    if dtype not in _ELEM:
        raise ValueError(f"Q: float32 or bfloat16 is needed, not {dtype}")
    qp, qs = _heads(Q, "Q", B, Hq, cache.D, dtype, dev)
    if out.shape != Q.shape or out.dtype is not dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out: a contiguous tensor of Q's shape, type and device is needed")
    if lse is not None and (lse.dtype is not _FP32 or lse.shape != (B, Hq) or lse.device != dev
                            or not lse.is_contiguous()):
        raise ValueError(f"lse: a contiguous float32 tensor [{B}, {Hq}] on {dev} is needed")
    tp, ts, rows, width = _table(table, dev)
    if rows != B:
        raise ValueError(f"table: {B} rows are needed, not {rows}")
    wp, wn = _room(workspace, dev)
    _on(dev, _L.lsa_paged_attn,
        (qp, _ELEM[dtype], qs, cache._ref, tp, ts, width, _i32(seq_len, "seq_len", dev, B), B, Hq, window,
         D ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), wp, wn,
         _err_word(err, dev)), "lsa_paged_attn", stream)


ROPE_KINDS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_frequencies(rot_dim, base=10000.0, kind="plain", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    """(frequencies float64 [rot_dim / 2] on the host, mscale) of a plain or scaled rotation (lsa_rope_frequencies)."""
    _need(kind in ROPE_KINDS, f"kind: one of {', '.join(ROPE_KINDS)} is needed, not {kind!r}")
    _fits(rot_dim, "rot_dim")
    freq, m = torch.empty(max(1, rot_dim // 2), dtype=torch.float64), ctypes.c_float()
    _check(_L.lsa_rope_frequencies(ROPE_KINDS[kind], rot_dim, base, factor, orig_len, beta_fast, beta_slow,
                                   freq.data_ptr(), ctypes.byref(m)), "lsa_rope_frequencies")
    return freq, float(m.value)


class Rope:
    """A rotation by position (lsa_rope in lsa.h).  freq: contiguous float64 [rot_dim / 2] on the device, radians per
    position (rope_frequencies gives plain and scaled ones)."""

    def __init__(self, freq, interleaved=False, inverse=False, mscale=1.0):
        _need(freq.dtype == torch.float64 and freq.dim() == 1 and freq.is_contiguous(),
              "freq: a contiguous float64 vector is needed")
        _need(mscale > 0, "mscale must be positive")
        self.freq, self.device = freq, freq.device if freq.numel() else None
        self.desc = RopeDesc(_ptr(freq), 2 * freq.numel(), int(interleaved), int(inverse), mscale)
        self._ref = ctypes.byref(self.desc)


def _weight(w, name, D, dtype, device):
    if w is None:
        return None
    if w.dtype is not dtype or w.shape != (D,) or not w.is_contiguous() or w.device != device:
        raise ValueError(f"{name}: a contiguous tensor [{D}] of {dtype} on {device} is needed")
    return w.data_ptr()


def qk_norm_rope(q, k=None, v=None, *, q_out, k_out=None, q_weight=None, k_weight=None, eps=1e-6, pos=None, rope=None,
                 cache=None, table=None, seq=None, at=None, err=None, stream=None):
    """Norm and rotation of a step's query and key heads, and the append of keys and values to a PageCache
    (lsa_qk_norm_rope).

    q [T, Hq, D], k and v [T, Hkv, D] (any stride between tokens; parts of one projection's output are fine); q_out,
    k_out likewise, or q and k themselves.  q_weight, k_weight [D]: norm weights, None: no norm.  pos int32 [T] with
    rope.  With cache: token t becomes entry at[t] of table row seq[t] (row t if seq is None).
    """
    dev, dtype = q.device, q.dtype
    T, Hq, D = q.shape
    if dtype not in _ELEM:
        raise ValueError(f"q: float32 or bfloat16 is needed, not {dtype}")
    Hkv, kp, ks, kop, kos, vp, vs, tp, ts, rows, width = 0, None, 0, None, 0, None, 0, None, 0, 0, 0
    qp, qs = _heads(q, "q", T, Hq, D, dtype, dev)
    qop, qos = _heads(q_out, "q_out", T, Hq, D, dtype, dev)
    if k is not None:
        Hkv = k.shape[1]
        kp, ks = _heads(k, "k", T, Hkv, D, dtype, dev)
    if k_out is not None:
        kop, kos = _heads(k_out, "k_out", T, Hkv, D, dtype, dev)
    if v is not None:
        vp, vs = _heads(v, "v", T, Hkv, D, dtype, dev)
    if rope is not None and rope.device != dev and rope.device is not None:
        raise ValueError(f"rope: freq on {dev} is needed")
    if cache is not None:
        if cache.device != dev or table is None or at is None:
            raise ValueError(f"cache: one on {dev}, with table and at, is needed")
        tp, ts, rows, width = _table(table, dev)
    _on(dev, _L.lsa_qk_norm_rope,
        (qp, qs, qop, qos, kp, ks, kop, kos, vp, vs, _ELEM[dtype], T, Hq, Hkv, D,
         _weight(q_weight, "q_weight", D, dtype, dev), _weight(k_weight, "k_weight", D, dtype, dev), eps,
         None if pos is None else _i32(pos, "pos", dev, T), None if rope is None else rope._ref,
         None if cache is None else cache._ref, tp, ts, rows, width,
         None if seq is None else _i32(seq, "seq", dev, T), None if at is None else _i32(at, "at", dev, T),
         _err_word(err, dev)), "lsa_qk_norm_rope", stream)


class PageTable:
    """The books of a cache's pages (lsa_page_table in lsa.h): table int32 [n_rows, max_pages], len int32 [n_rows] and
    refs int32 [n_pages], contiguous, on one device."""

    def __init__(self, table, length, refs, page_size):
        _need(table.dim() == 2 and refs.dim() == 1, "table: [n_rows, max_pages] and refs: [n_pages] are needed")
        self.table, self.len, self.refs, self.page_size = table, length, refs, int(page_size)
        _fits(self.page_size, "page_size")
        self.device = table.device
        self.n_rows, self.max_pages = table.shape
        self.n_pages = refs.numel()
        self.desc = PageTableDesc(_i32(table, "table", self.device, *table.shape),
                                  _i32(length, "length", self.device, self.n_rows),
                                  _i32(refs, "refs", self.device, self.n_pages), self.n_rows, self.max_pages,
                                  self.page_size, self.n_pages)
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, n_rows, max_pages, n_pages, page_size, device="cuda"):
        """Books without a held page."""
        return cls(torch.full((n_rows, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_rows, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device), page_size)


def page_grow(pages, add, err=None, stream=None):
    """Row r of `pages` becomes add[r] entries longer and takes the pages that needs (lsa_page_grow)."""
    dev = pages.device
    _on(dev, _L.lsa_page_grow, (pages._ref, _i32(add, "add", dev, pages.n_rows), _err_word(err, dev)),
        "lsa_page_grow", stream)


def page_fork(pages, src, dst, copy_src, copy_dst, err=None, stream=None):
    """Row dst[i] becomes a copy of row src[i]; (copy_src, copy_dst): the pages to copy, -1 for none (lsa_page_fork)."""
    dev, n = pages.device, src.numel()
    _on(dev, _L.lsa_page_fork,
        (pages._ref, _i32(src, "src", dev, n), _i32(dst, "dst", dev, n), n, _i32(copy_src, "copy_src", dev, n),
         _i32(copy_dst, "copy_dst", dev, n), _err_word(err, dev)), "lsa_page_fork", stream)


def page_free(pages, rows, err=None, stream=None):
    """The rows give back their pages and become empty (lsa_page_free)."""
    dev, n = pages.device, rows.numel()
    _on(dev, _L.lsa_page_free, (pages._ref, _i32(rows, "rows", dev, n), n, _err_word(err, dev)), "lsa_page_free", stream)


def page_compact_workspace_size(n_pages) -> int:
    return int(_L.lsa_page_compact_workspace_size(n_pages))


def page_compact(pages, table_out, refs_out, move_src, move_dst, n_moves, workspace, stream=None):
    """Packs the held pages to the pool's front (lsa_page_compact); the moves go to page_copy of each layer's cache."""
    dev, n = pages.device, pages.n_pages
    wp, wn = _room(workspace, dev)
    _on(dev, _L.lsa_page_compact,
        (pages._ref, _i32(table_out, "table_out", dev, pages.n_rows, pages.max_pages),
         _i32(refs_out, "refs_out", dev, n), _i32(move_src, "move_src", dev, n), _i32(move_dst, "move_dst", dev, n),
         _i32(n_moves, "n_moves", dev, 1), wp, wn), "lsa_page_compact", stream)


def page_copy(cache, src, dst, count=None, err=None, stream=None):
    """Copies pages src[i] -> dst[i] of a PageCache (lsa_page_copy), the first `count` of them where that is given."""
    dev, n = cache.device, src.numel()
    _on(dev, _L.lsa_page_copy,
        (cache._ref, _i32(src, "src", dev, n), _i32(dst, "dst", dev, n), n,
         None if count is None else _i32(count, "count", dev, 1), _err_word(err, dev)), "lsa_page_copy", stream)


# ----------------------------------------------------------- decode context

class Context:
    """Owns an lsa_ctx: the tau-cadence decode loop over device-resident keys and a pinned cold pool.

    The caller keeps `keys`, `k_scale` and `cold_host` alive for the context's lifetime.
    """

    def __init__(self, *, B, H, d, q_dtype, k_dtype, Hq, D, attn_dtype, topk, seq_off_host, keys, k_scale,
                 cold_host, row_bytes, kv_row_stride, k_off, v_off, kept_capacity, tau=64, scale=0.0,
                 full_fetch=False, window=0, hca_rows=None, hca_off_host=None, layers=None, lookahead=0):
        """window / hca_rows / hca_off_host: the always-resident context merged into the attention set
        (see lsa_attn_set_merge); hca_rows is a host or device tensor of HCA rows in the cold-pool row format.
        layers: [(keys, k_scale), ...] of indexer layers 1 .. L-1 (layer 0 is keys / k_scale) for the OR-mode
        union in the cadence; steps then take q [L, B, H, d] and w [L, B, H].
        lookahead: predict each window's kept set this many steps ahead and fetch it meanwhile (see lsa.h)."""
        self._seq_off = torch.as_tensor(seq_off_host, dtype=torch.int64).contiguous()
        self._hca_off = None if hca_off_host is None else torch.as_tensor(hca_off_host, dtype=torch.int64).contiguous()
        n_total = int(self._seq_off[-1])
        self.params = Params(B, H, d, DTYPE[q_dtype], DTYPE[k_dtype], Hq, D, DTYPE[attn_dtype], topk, tau,
                             float(scale), n_total, self._seq_off.data_ptr(), _ptr(keys), _ptr(k_scale),
                             _ptr(cold_host), row_bytes, kv_row_stride, k_off, v_off, kept_capacity,
                             int(bool(full_fetch)), int(window), _ptr(hca_rows),
                             None if self._hca_off is None else self._hca_off.data_ptr())
        self.params.lookahead = int(lookahead)
        self.n_layers = 1
        if layers:
            self.n_layers = 1 + len(layers)
            self._karr = (P * len(layers))(*[_ptr(k) for k, _ in layers])
            self._sarr = (P * len(layers))(*[_ptr(s) for _, s in layers])
            self.params.n_layers = self.n_layers
            self.params.k_dev_layers = ctypes.cast(self._karr, P)
            self.params.k_scale_layers = ctypes.cast(self._sarr, P) if k_scale is not None else None
        self._keep = (keys, k_scale, cold_host, layers)
        h = P()
        _check(_L.lsa_ctx_create(ctypes.byref(self.params), ctypes.byref(h)), "lsa_ctx_create")
        self.handle = h
        self.B, self.topk, self.n_total, self.kept_capacity = B, topk, n_total, kept_capacity
        self.row_bytes = row_bytes

    def close(self):
        if self.handle:
            _check(_L.lsa_ctx_destroy(self.handle), "lsa_ctx_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def step(self, t, q, w, Q, out, lse=None, stream=None):
        _check(_L.lsa_decode_step(self.handle, t, _ptr(q), _ptr(w), _ptr(Q), _ptr(out), _ptr(lse), _stream(stream)),
               "lsa_decode_step")

    def step_host(self, t, q_host, w_host, Q_host, out_host, lse_host=None, stream=None):
        _check(_L.lsa_decode_step_host(self.handle, t, _ptr(q_host), _ptr(w_host), _ptr(Q_host), _ptr(out_host),
                                       _ptr(lse_host), _stream(stream)), "lsa_decode_step_host")

    def view(self) -> View:
        v = View()
        _check(_L.lsa_ctx_get_view(self.handle, ctypes.byref(v)), "lsa_ctx_get_view")
        return v

    def set_graphs(self, on: bool):
        _check(_L.lsa_ctx_set_graphs(self.handle, int(on)), "lsa_ctx_set_graphs")

    def set_timing(self, on: bool):
        _check(_L.lsa_ctx_set_timing(self.handle, int(on)), "lsa_ctx_set_timing")

    def stage_times(self):
        ms = (ctypes.c_double * N_STAGES)()
        calls = (i64 * N_STAGES)()
        _check(_L.lsa_ctx_stage_times(self.handle, ms, calls), "lsa_ctx_stage_times")
        return {STAGES[i]: (ms[i], calls[i]) for i in range(N_STAGES)}

    def reset_counters(self):
        _check(_L.lsa_ctx_reset_counters(self.handle), "lsa_ctx_reset_counters")

    def launches(self) -> int:
        return int(_L.lsa_ctx_launches(self.handle))

    def flush_cache(self, stream=None):
        """Empty the hot-buffer cache: the next refresh or prediction fetches every kept row."""
        _check(_L.lsa_ctx_flush_cache(self.handle, _stream(stream)), "lsa_ctx_flush_cache")

    def fetched(self) -> int:
        """Rows the last refresh fetched from the cold pool (synchronises the device)."""
        return int(device_view(self.view().fetched, 1, torch.int64).item())


_cudart = None


def device_view(ptr: int, numel: int, dtype: torch.dtype) -> torch.Tensor:
    """Copy `numel` elements at a device address owned by a context into a new tensor (for inspection).

    Synchronises the device first; uses the CUDA runtime torch already loaded.
    """
    global _cudart
    if _cudart is None:
        _cudart = ctypes.CDLL("libcudart.so.12")
        _cudart.cudaMemcpy.restype = ctypes.c_int
        _cudart.cudaMemcpy.argtypes = [P, P, sz, ctypes.c_int]
    out = torch.empty(numel, dtype=dtype, device="cuda")
    if numel:
        torch.cuda.synchronize()
        rc = _cudart.cudaMemcpy(out.data_ptr(), ptr, numel * out.element_size(), 3)  # device to device
        if rc != 0:
            raise RuntimeError(f"cudaMemcpy failed with error {rc}")
    return out
