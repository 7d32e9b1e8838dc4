"""Mixture-of-Gaussians (MoG) decode attention for NVIDIA GB300.

A thin ctypes binding of ``libmog.so`` (the CUDA kernels and the C ABI in
``include/mog.h``).  This module only marshals arguments: device memory comes from
PyTorch tensors, streams from ``torch.cuda.current_stream()``, and every step of the
build and decode runs in the library's kernels.  There is no CPU fallback: if the
library is missing or fails to load, every call raises.

Sources: "Iceberg Attention: Sublinear Long-Context Decoding with Mixture-of-Gaussians"
(Abstract) and the newx.sg page on retrieval-completion attention (Abstract).
"""
from __future__ import annotations

import ctypes as C
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmog.so")

MOG_OK = 0
FLAG_UNION_EXACT = 1  # MOG_FLAG_UNION_EXACT in mog.h
FLAG_SLIDING = 2      # MOG_FLAG_SLIDING in mog.h
FLAG_GROUP_SELECT = 4  # MOG_FLAG_GROUP_SELECT in mog.h
FLAG_BF16_SUMMARIES = 8  # MOG_FLAG_BF16_SUMMARIES in mog.h
FLAG_FP8_SUMMARIES = 16  # MOG_FLAG_FP8_SUMMARIES in mog.h
FLAG_KMEANSPP = 32       # MOG_FLAG_KMEANSPP in mog.h
RESIDUAL_FEATURE_MAP = 2  # MOG_RESIDUAL_FEATURE_MAP in mog.h
FM_FEATURES = 32          # MOG_FM_FEATURES in mog.h
STATUS = ["MOG_OK", "MOG_ERR_INVALID_ARG", "MOG_ERR_SHAPE", "MOG_ERR_ARENA_TOO_SMALL",
          "MOG_ERR_CUDA", "MOG_ERR_DEVICE_CHECK", "MOG_ERR_TIMEOUT", "MOG_ERR_NOT_IMPLEMENTED",
          "MOG_ERR_CAPACITY"]


class MogError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        name = STATUS[code] if 0 <= code < len(STATUS) else f"status {code}"
        super().__init__(f"{where}: {name}" + (f" ({detail})" if detail else ""))


class Params(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "batch", "h_kv", "h_q", "d", "n_cap", "n_clusters", "n_sub", "top_c", "top_s",
        "n_sink", "n_recent", "iters_l1", "iters_l2", "score_mode", "residual", "flags")]


class KV(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("stride_b", C.c_int64),
                ("stride_h", C.c_int64), ("stride_n", C.c_int64), ("block_table", C.c_void_p),
                ("page_rows", C.c_int32), ("pages_per_seq", C.c_int32)]


class PagedKV:
    """A paged bf16 KV cache: page pools K, V of shape [pages, H_kv, page_rows, d]
    (heads_first) or [pages, page_rows, H_kv, d], and an int32 block table [B, pages_per_seq]
    on the device (page of position n of sequence b: block_table[b, n // page_rows]).
    Pass it as K (with V=None) wherever a cache is taken."""

    def __init__(self, K, V, block_table, page_rows, heads_first=True):
        torch = _torch()
        _check_pools(K, V)
        if not (K.is_cuda and V.is_cuda):
            raise ValueError("page pools must be CUDA tensors")
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 tensor [B, pages_per_seq]")
        self.K, self.V, self.block_table, self.page_rows = K, V, block_table, page_rows
        self.heads_first = heads_first
        self.h_kv = K.shape[1] if heads_first else K.shape[2]
        self.device = K.device
        self._cache = None  # (made when a call first needs it)
        self._checked = K, V

    def struct(self) -> KV:
        K, V = self.K, self.V
        if self._checked[0] is not K or self._checked[1] is not V:  # (set anew)
            _check_pools(K, V)
            self._checked = K, V
        sh, sn = (K.stride(1), K.stride(2)) if self.heads_first else (K.stride(2), K.stride(1))
        return KV(K.data_ptr(), self.V.data_ptr(), K.stride(0), sh, sn, self.block_table.data_ptr(),
                  self.page_rows, self.block_table.shape[1])


class Cache(C.Structure):
    _fields_ = [("type", C.c_int32), ("n_cap", C.c_int32), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("stride_b", C.c_int64),
                ("stride_h", C.c_int64), ("stride_n", C.c_int64), ("scale_b", C.c_int64),
                ("scale_h", C.c_int64), ("scale_n", C.c_int64), ("block_table", C.c_void_p),
                ("page_rows", C.c_int32), ("pages_per_seq", C.c_int32), ("n_pages", C.c_int32)]


class DiffParams(C.Structure):
    _fields_ = [("lam", C.c_void_p), ("gamma", C.c_void_p), ("lam_heads", C.c_int32),
                ("lambda_init", C.c_float), ("eps", C.c_float)]


class PagePoolDesc(C.Structure):
    _fields_ = [("base", C.c_void_p), ("page_stride", C.c_int64), ("page_bytes", C.c_int64)]


class Pages(C.Structure):
    _fields_ = [("n_pages", C.c_int32), ("page_rows", C.c_int32), ("batch", C.c_int32),
                ("pages_per_seq", C.c_int32), ("block_table", C.c_void_p), ("lengths", C.c_void_p),
                ("refs", C.c_void_p), ("work", C.c_void_p), ("work_bytes", C.c_size_t),
                ("pools", C.POINTER(PagePoolDesc)), ("n_pools", C.c_int32)]


def _strides(t):
    """Strides of a tensor's first three dims, 0 where there is only one entry (its stride may
    be anything)."""
    return [st if n > 1 else 0 for n, st in zip(t.shape[:3], t.stride())]


def _check_rows8(K, V, k_scale, v_scale):
    torch = _torch()
    for t in (K, V):
        if t.dtype != torch.float8_e4m3fn or t.dim() != 4 or t.stride(3) != 1 or not t.is_cuda:
            raise ValueError("K and V must be CUDA float8_e4m3fn tensors with 4 dims, last contiguous")
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != K.shape[:3] or t.device != K.device:
            raise ValueError("the scales must be float32 tensors of K's first three dims on its device")
    if K.shape != V.shape or K.stride() != V.stride() or V.device != K.device:
        raise ValueError("K and V must share shape, strides and device")
    if k_scale.stride() != v_scale.stride():
        raise ValueError("the scales must share strides")
    if K.shape[3] != 128:
        raise ValueError("the last dim of K and V must be 128")


class _Fixed:
    """An object whose attributes stay as they were made: its C structure holds their addresses."""

    def __setattr__(self, name, value):
        if "_made" in self.__dict__:
            raise AttributeError(f"a {type(self).__name__} is fixed once it is made: {name} cannot be set")
        object.__setattr__(self, name, value)


class KV8(_Fixed):
    """A contiguous e4m3 KV cache: codes K, V float8_e4m3fn [B, H_kv, n_cap, 128] and a scale
    per row, k_scale, v_scale float32 [B, H_kv, n_cap] (value = scale * code).  Pass it as K
    (with V=None) to dense_decode, diff_decode and kv_store.  The tensors are fixed once it
    is made."""

    def __init__(self, K, V, k_scale, v_scale):
        _check_rows8(K, V, k_scale, v_scale)
        self.K, self.V, self.k_scale, self.v_scale = K, V, k_scale, v_scale
        self.batch, self.h_kv, self.device = K.shape[0], K.shape[1], K.device
        self.positions = K.shape[2]
        self.cache = Cache(1, K.shape[2], K.data_ptr(), V.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                           *_strides(K)[:2], K.stride(2), *_strides(k_scale), None, 0, 0, 0)
        self._made = True


class PagedKV8(_Fixed):
    """A paged e4m3 KV cache: page pools K, V float8_e4m3fn [pages, H_kv, page_rows, 128]
    (heads_first) or [pages, page_rows, H_kv, 128], a scale per row, k_scale, v_scale float32
    of the pools' first three dims, and an int32 block table [B, pages_per_seq] on the device.
    Pass it as K (with V=None) to dense_decode, diff_decode and kv_store.  The tensors are
    fixed once it is made; the block table's entries may change between calls."""

    def __init__(self, K, V, k_scale, v_scale, block_table, page_rows, heads_first=True):
        _check_rows8(K, V, k_scale, v_scale)
        _check_table(block_table, K)
        if K.shape[2 if heads_first else 1] != page_rows:
            raise ValueError("page_rows must be the pools' rows per page")
        self.K, self.V, self.k_scale, self.v_scale = K, V, k_scale, v_scale
        self.block_table, self.page_rows, self.heads_first = block_table, page_rows, heads_first
        self.batch, self.h_kv = block_table.shape[0], K.shape[1 if heads_first else 2]
        self.positions, self.device = block_table.shape[1] * page_rows, K.device
        h, n = (1, 2) if heads_first else (2, 1)
        ks, ss = _strides(K), _strides(k_scale)
        self.cache = Cache(1, 0, K.data_ptr(), V.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), ks[0], ks[h],
                           ks[n], ss[0], ss[h], ss[n], block_table.data_ptr(), page_rows, block_table.shape[1],
                           K.shape[0])
        self._made = True


def _check_table(block_table, K):
    torch = _torch()
    if (block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous()
            or block_table.device != K.device):
        raise ValueError("block_table must be a contiguous int32 tensor [B, pages_per_seq] on the pools' device")


def _check_pools(K, V):
    bf16, st = _torch().bfloat16, K.stride()
    if K.dtype is not bf16 or V.dtype is not bf16 or len(st) != 4 or st[3] != 1:
        raise ValueError("page pools must be bf16 tensors with 4 dims, last contiguous")
    if K.shape != V.shape or st != V.stride():
        raise ValueError("K and V pools must share shape and strides")


def _paged_cache(P):
    k, v, t, rows = P.K, P.V, P.block_table, P.page_rows
    _check_pools(k, v)
    _check_table(t, k)
    shape, st = k.shape, k.stride()
    h, n = (1, 2) if P.heads_first else (2, 1)
    if v.device != k.device or shape[3] != 128 or shape[n] != rows:
        raise ValueError("page pools must share a device and hold page_rows rows of 128")
    per = t.shape[1]
    c = Cache(0, 0, k.data_ptr(), v.data_ptr(), None, None, st[0] if shape[0] > 1 else 0, st[h] if shape[h] > 1 else 0,
              st[n], 0, 0, 0, t.data_ptr(), rows, per, shape[0])
    return c, t.shape[0], shape[h], per * rows, k.device


def _cache(K, V):
    """(mog_cache, batch, KV heads, positions, device) of a KV8, a PagedKV8, a PagedKV or two
    bf16 tensors [B, H_kv, n_cap, 128]."""
    if isinstance(K, (KV8, PagedKV8)):
        return K.cache, K.batch, K.h_kv, K.positions, K.device
    if isinstance(K, PagedKV):
        k, v, t = K.K, K.V, K.block_table
        of = (k.data_ptr(), v.data_ptr(), t.data_ptr(), k.shape, v.shape, t.shape, k.stride(), v.stride(), t.stride(),
              K.page_rows, K.heads_first)
        made = K._cache  # its mog_cache, with what it was made of: the attributes may be set anew
        if made is None or made[2] is not k or made[3] is not v or made[4] is not t or made[0] != of:
            made = K._cache = of, _paged_cache(K), k, v, t
        return made[1]
    torch = _torch()
    if V is None:
        raise ValueError("this call takes K and V tensors, or a PagedKV, KV8 or PagedKV8 as K")
    shape, st, dev = K.shape, K.stride(), K.device
    if (K.dtype is not torch.bfloat16 or V.dtype is not torch.bfloat16 or len(shape) != 4 or shape[3] != 128
            or st[3] != 1 or V.shape != shape or V.stride() != st or dev.type != "cuda" or V.device != dev):
        raise ValueError("K and V must be CUDA bf16 tensors [B, H_kv, n_cap, 128] of one shape, strides and device, "
                         "last dim contiguous")
    B, H, n = shape[:3]
    return Cache(0, n, K.data_ptr(), V.data_ptr(), None, None, st[0] if B > 1 else 0, st[1] if H > 1 else 0, st[2]), B, H, n, dev


class Layout(C.Structure):
    _fields_ = ([(n, C.c_int32) for n in ("units", "c_max", "l_max", "n_cap", "d", "group",
                                           "top_c", "top_s")] +
                [(n, C.c_int64) for n in ("unit_info", "n_now", "perm", "sub_off",
                                           "sub_off_stride", "cl_n", "cl_ms", "cl_vbar", "sub_n",
                                           "sub_ms", "sub_vbar", "l1_assign", "status",
                                           "l1_steps", "fallback", "cl_ms16", "sub_ms16", "cl_ms8",
                                           "sub_ms8", "pp_idx", "fm_z", "fm_t")])


class TraceLayout(C.Structure):
    _fields_ = ([(n, C.c_int32) for n in ("units", "iters_l1", "iters_l2", "c_max", "l_max", "d")] +
                [(n, C.c_int64) for n in ("n_mid", "l1_cent", "l1_assign", "l2_cent", "l2_assign",
                                           "l2_steps", "bytes")])


_lib = None
_P = C.c_void_p
_SIGS = {
    "mog_status_string": (C.c_char_p, [C.c_int]),
    "mog_last_error": (C.c_char_p, []),
    "mog_arena_bytes": (C.c_int, [_P, _P, _P]),
    "mog_build": (C.c_int, [_P, _P, _P, _P, _P, C.c_size_t, _P, _P]),
    "mog_build_from_partition": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P, _P]),
    "mog_sub_off_stride": (C.c_int, [_P, _P, _P]),
    "mog_trace_layout_of": (C.c_int, [_P, _P, _P]),
    "mog_build_traced": (C.c_int, [_P, _P, _P, _P, _P, C.c_size_t, _P, C.c_size_t, _P, _P]),
    "mog_build_seeded": (C.c_int, [_P, _P, _P, _P, _P, _P, C.c_size_t, _P, C.c_size_t, _P, _P]),
    "mog_decode": (C.c_int, [_P, _P, _P, _P]),
    "mog_decode_ex": (C.c_int, [_P, _P, _P, _P, _P, _P]),
    "mog_decode_phased": (C.c_int, [_P, _P, _P, _P, _P, _P, _P]),
    "mog_append": (C.c_int, [_P, _P, _P, _P]),
    "mog_recluster": (C.c_int, [_P, _P]),
    "mog_feature_map": (C.c_int, [_P, _P, _P]),
    "mog_get_layout": (C.c_int, [_P, _P]),
    "mog_sync_status": (C.c_int, [_P, _P]),
    "mog_decode_splits": (C.c_int, [_P, _P]),
    "mog_destroy": (None, [_P]),
    "dense_decode_scratch_bytes": (C.c_int, [C.c_int32] * 5 + [_P]),
    "dense_decode": (C.c_int, [_P, _P, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                               _P, _P, _P, C.c_size_t, _P]),
    "dense_decode_noalloc": (C.c_int, [_P, _P, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                       C.c_int32, _P, _P, _P]),
    "mog_kmeans_assign_scratch_bytes": (C.c_int, [C.c_int32, C.c_int32, C.c_int32, _P]),
    "mog_kmeans_assign": (C.c_int, [_P, C.c_int64, C.c_int32, _P, C.c_int32, C.c_int32, _P, _P,
                                    C.c_size_t, _P, _P]),
    "mog_kmeans_assign_segments": (C.c_int, [_P, C.c_int64, _P, _P, C.c_int32, _P, C.c_int32,
                                             C.c_int32, _P, _P]),
    "dense_decode8_scratch_bytes": (C.c_int, [C.c_int32] * 5 + [_P]),
    "dense_decode8": (C.c_int, [_P, _P] + [C.c_int32] * 5 + [_P, _P, C.c_int32, _P, C.c_size_t, _P]),
    "mog_diff_decode_scratch_bytes": (C.c_int, [C.c_int32] * 5 + [_P]),
    "mog_diff_decode": (C.c_int, [_P, _P] + [C.c_int32] * 5 + [_P, _P, _P, C.c_int32, _P, C.c_size_t, _P]),
    "mog_kv_store": (C.c_int, [_P] + [C.c_int32] * 4 + [_P] * 4 + [C.c_int64] * 3 + [_P]),
    "mog_pages_work_bytes": (C.c_int, [C.c_int32, C.c_int32, _P]),
    "mog_pages_assign": (C.c_int, [_P, _P, _P]),
    "mog_pages_grow": (C.c_int, [_P, _P, _P, _P, _P]),
    "mog_pages_compact": (C.c_int, [_P, _P]),
    "mog_pages_status": (C.c_int, [_P, _P]),
    "mog_check_bounded_wait": (C.c_int, [C.c_int32, C.c_int32, _P, _P]),
}


def lib():
    """Load libmog.so (built in-tree by ``build.py``).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmog.so is not built ({LIB_PATH}); run "
                               "`python -m serving_mog_decode_gb300.build` first")
        l = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(rc: int, where: str):
    if rc != MOG_OK:
        detail = lib().mog_last_error().decode() if rc == 4 else ""
        raise MogError(rc, where, detail)


def _torch():
    import torch
    return torch


def _stream(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else None


def _kv(K, V):
    """KV descriptor of bf16 tensors [B, H_kv, n_cap, d] (last dim contiguous), or of a
    PagedKV passed as K."""
    if isinstance(K, PagedKV):
        return K.struct()
    torch = _torch()
    if isinstance(K, (KV8, PagedKV8)) or V is None:
        raise ValueError("this call takes bf16 K and V tensors, or a PagedKV as K")
    for t in (K, V):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(3) != 1 or not t.is_cuda:
            raise ValueError("K and V must be CUDA bf16 tensors [B, H_kv, n_cap, d], last dim contiguous")
    if K.stride() != V.stride() or K.shape != V.shape:
        raise ValueError("K and V must share shape and strides")
    return KV(K.data_ptr(), V.data_ptr(), K.stride(0), K.stride(1), K.stride(2))


def make_params(batch, h_kv, h_q, n_cap, *, d=128, n_clusters=0, n_sub=0, top_c=8, top_s=8,
                n_sink=4, n_recent=256, iters_l1=10, iters_l2=10, score_mode=0, residual=1,
                union_exact=0, sliding=0, group_select=0, bf16_summaries=0, fp8_summaries=0,
                kmeanspp=0):
    """mog_params for a batch of `batch` sequences with h_kv KV heads and h_q query heads
    (d = 128), a KV cache of n_cap positions.  n_clusters / n_sub = 0 pick round(sqrt N)
    and ceil(log2 N) per sequence; top_c clusters and top_s subclusters per chosen cluster
    are attended exactly, with n_sink sink and n_recent recent anchors.  The flags select
    the variants: union_exact (every head of a KV group attends the union of the group's
    chosen rows), sliding (a fixed recent window whose leaving keys join the clusters),
    group_select (one selection per KV group by the log-sum-exp of its heads' scores),
    bf16_summaries or fp8_summaries (scores and residual terms from the summaries rounded to
    bf16, or to fp8 e4m3; not both), kmeanspp (first-level k-means++ seeds; build() then
    needs the draws)."""
    return Params(batch, h_kv, h_q, d, n_cap, n_clusters, n_sub, top_c, top_s, n_sink,
                  n_recent, iters_l1, iters_l2, score_mode, residual,
                  (FLAG_UNION_EXACT if union_exact else 0) | (FLAG_SLIDING if sliding else 0)
                  | (FLAG_GROUP_SELECT if group_select else 0)
                  | (FLAG_BF16_SUMMARIES if bf16_summaries else 0)
                  | (FLAG_FP8_SUMMARIES if fp8_summaries else 0)
                  | (FLAG_KMEANSPP if kmeanspp else 0))


def arena_bytes(params: Params, lengths_host) -> int:
    import numpy as np
    lh = np.ascontiguousarray(lengths_host, np.int32)
    out = C.c_size_t(0)
    _check(lib().mog_arena_bytes(C.byref(params), lh.ctypes.data_as(_P), C.byref(out)),
           "mog_arena_bytes")
    return out.value


class Handle:
    """A built MoG index over a KV cache.  Owns (references) the arena tensor; the KV
    tensors must stay alive and unmoved while the handle is used."""

    def __init__(self, ptr, arena, params, K, V, lengths_dev, lengths_host):  # K may be a PagedKV
        self._h = ptr
        self.arena = arena
        self.params = params
        self.K, self.V = K, V
        self.lengths_dev = lengths_dev
        self.lengths_host = lengths_host

    def __del__(self):
        if getattr(self, "_h", None):
            try:
                lib().mog_destroy(self._h)
            except Exception:
                pass
            self._h = None

    @property
    def group(self):
        return self.params.h_q // self.params.h_kv

    def decode(self, q, out=None, sel_in=None, sel_out=None, stream=None):
        torch = _torch()
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        if sel_in is None and sel_out is None:
            rc = lib().mog_decode(self._h, _ptr(q), _ptr(out), _stream(stream))
        else:
            rc = lib().mog_decode_ex(self._h, _ptr(q), _ptr(out), _ptr(sel_in), _ptr(sel_out),
                                     _stream(stream))
        _check(rc, "mog_decode")
        return out

    def decode_phased(self, q, out, events, sel_out=None, stream=None):
        """Decode with four torch.cuda.Event objects recorded around the three kernels."""
        for e in events:       # torch creates the CUDA event on first record
            if not e.cuda_event:
                e.record()
        arr = (C.c_void_p * 4)(*[e.cuda_event for e in events])
        _check(lib().mog_decode_phased(self._h, _ptr(q), _ptr(out), None, _ptr(sel_out), arr,
                                       _stream(stream)), "mog_decode_phased")
        return out

    def append(self, k_new, v_new, stream=None):
        _check(lib().mog_append(self._h, _ptr(k_new), _ptr(v_new), _stream(stream)), "mog_append")

    def recluster(self, stream=None):
        """Rebuild the partition and summaries over the grown sequences (mog_recluster)."""
        _check(lib().mog_recluster(self._h, _stream(stream)), "mog_recluster")

    def feature_map(self, omega, stream=None):
        """The feature-map summary for residual = 2 (mog_feature_map): omega, float32
        [FM_FEATURES, 128] frequencies drawn N(0, I), on the cache's device."""
        torch = _torch()
        om = torch.as_tensor(omega, dtype=torch.float32, device=self.arena.device).contiguous()
        if tuple(om.shape) != (FM_FEATURES, 128):
            raise ValueError(f"omega must be [{FM_FEATURES}, 128]")
        self._omega = om   # kept alive until the copy has run
        _check(lib().mog_feature_map(self._h, _ptr(om), _stream(stream)), "mog_feature_map")

    def splits(self) -> int:
        v = C.c_int32(0)
        _check(lib().mog_decode_splits(self._h, C.byref(v)), "mog_decode_splits")
        return v.value

    def layout(self) -> Layout:
        lay = Layout()
        _check(lib().mog_get_layout(self._h, C.byref(lay)), "mog_get_layout")
        return lay

    def sync_status(self, stream=None) -> int:
        return lib().mog_sync_status(self._h, _stream(stream))

    def array(self, name: str, dtype, shape):
        """A view of one arena array (see mog_layout) as a torch tensor."""
        torch = _torch()
        off = getattr(self.layout(), name)
        n = 1
        for s in shape:
            n *= s
        itemsize = torch.empty((), dtype=dtype).element_size()
        return self.arena[off:off + n * itemsize].view(dtype).view(*shape)


class Trace:
    """The build trace of mog_build_traced (see mog_trace_layout in mog.h) as torch views:
    l1_cent [U, T1, c_max, d], l1_assign [U, T1, n_mid], l2_cent [U, c_max, T2, l_max, d],
    l2_assign [U, T2, n_mid], l2_steps [U, c_max]."""

    def __init__(self, buf, lay: TraceLayout):
        torch = _torch()
        self.buf, self.layout = buf, lay
        U, T1, T2, cm, lm, d, nm = (lay.units, lay.iters_l1, lay.iters_l2, lay.c_max, lay.l_max,
                                    lay.d, lay.n_mid)

        def view(off, dtype, shape):
            n = 1
            for x in shape:
                n *= x
            return buf[off:off + 4 * n].view(dtype).view(*shape)

        self.l1_cent = view(lay.l1_cent, torch.float32, (U, T1, cm, d))
        self.l1_assign = view(lay.l1_assign, torch.int32, (U, T1, nm))
        self.l2_cent = view(lay.l2_cent, torch.float32, (U, cm, T2, lm, d))
        self.l2_assign = view(lay.l2_assign, torch.int32, (U, T2, nm))
        self.l2_steps = view(lay.l2_steps, torch.int32, (U, cm))


def trace_layout(params: Params, lengths_host) -> TraceLayout:
    import numpy as np
    lh = np.ascontiguousarray(lengths_host, np.int32)
    lay = TraceLayout()
    _check(lib().mog_trace_layout_of(C.byref(params), lh.ctypes.data_as(_P), C.byref(lay)),
           "mog_trace_layout_of")
    return lay


def build(K, V, lengths, params: Params, stream=None, partition=None, trace=False, draws=None):
    """mog_build (or mog_build_from_partition when partition=(perm, sub_off) is given, or
    mog_build_traced when trace=True, which returns (handle, Trace)).  `lengths` is a host
    sequence of int; a device copy is made.  With the k-means++ flag, draws (float64
    [units, c_max] uniforms in [0, 1), c_max from trace_layout) go to mog_build_seeded."""
    import numpy as np
    torch = _torch()
    lh = np.ascontiguousarray(lengths, np.int32)
    ld = torch.from_numpy(lh.copy()).to(K.device)  # (a PagedKV has a device too)
    nbytes = arena_bytes(params, lh)
    arena = torch.empty(nbytes + 256, dtype=torch.uint8, device=K.device)
    off = (-arena.data_ptr()) % 256
    arena = arena[off:off + nbytes]
    kv = _kv(K, V)
    h = _P()
    if params.flags & FLAG_KMEANSPP:
        if draws is None:
            raise ValueError("k-means++ seeding needs draws (float64 [units, c_max] in [0, 1))")
        lay = trace_layout(params, lh)
        dr = torch.as_tensor(draws, dtype=torch.float64, device=K.device).contiguous()
        if dr.numel() != lay.units * lay.c_max:
            raise ValueError(f"k-means++ needs draws of shape [{lay.units}, {lay.c_max}]")
        tbuf = torch.empty(lay.bytes, dtype=torch.uint8, device=K.device) if trace else None
        rc = lib().mog_build_seeded(C.byref(kv), _ptr(ld), lh.ctypes.data_as(_P), C.byref(params),
                                    _ptr(dr), _ptr(arena), nbytes, _ptr(tbuf),
                                    lay.bytes if trace else 0, _stream(stream), C.byref(h))
        _check(rc, "mog_build_seeded")
        hd = Handle(h, arena, params, K, V, ld, lh)
        return (hd, Trace(tbuf, lay)) if trace else hd
    if trace:
        lay = trace_layout(params, lh)
        tbuf = torch.empty(lay.bytes, dtype=torch.uint8, device=K.device)
        rc = lib().mog_build_traced(C.byref(kv), _ptr(ld), lh.ctypes.data_as(_P), C.byref(params),
                                    _ptr(arena), nbytes, _ptr(tbuf), lay.bytes, _stream(stream),
                                    C.byref(h))
        _check(rc, "mog_build_traced")
        return Handle(h, arena, params, K, V, ld, lh), Trace(tbuf, lay)
    if partition is None:
        rc = lib().mog_build(C.byref(kv), _ptr(ld), lh.ctypes.data_as(_P), C.byref(params),
                             _ptr(arena), nbytes, _stream(stream), C.byref(h))
        _check(rc, "mog_build")
    else:
        perm, sub_off = partition
        rc = lib().mog_build_from_partition(C.byref(kv), _ptr(ld), lh.ctypes.data_as(_P),
                                            C.byref(params), _ptr(perm), _ptr(sub_off),
                                            _ptr(arena), nbytes, _stream(stream), C.byref(h))
        _check(rc, "mog_build_from_partition")
    return Handle(h, arena, params, K, V, ld, lh)


def sub_off_stride(params: Params, lengths_host) -> int:
    import numpy as np
    lh = np.ascontiguousarray(lengths_host, np.int32)
    v = C.c_int64(0)
    _check(lib().mog_sub_off_stride(C.byref(params), lh.ctypes.data_as(_P), C.byref(v)),
           "mog_sub_off_stride")
    return v.value


def dense_scratch_bytes(batch, h_kv, h_q, n_max, d=128) -> int:
    v = C.c_size_t(0)
    _check(lib().dense_decode_scratch_bytes(batch, h_kv, h_q, d, n_max, C.byref(v)),
           "dense_decode_scratch_bytes")
    return v.value


def _check_q_out(K, q, out):
    """q must be a contiguous CUDA bf16 [B, H_q, 128] on K's device and out a contiguous
    float32 tensor of q's shape on the same device: the kernels write B*H_q*128 floats."""
    torch = _torch()
    B = q.shape[0] if isinstance(K, PagedKV) else K.shape[0]
    if (q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[0] != B or q.shape[2] != 128
            or not q.is_contiguous() or q.device != K.device):
        raise ValueError("q must be a contiguous bf16 tensor [B, H_q, 128] on the cache's device")
    if (out.dtype != torch.float32 or tuple(out.shape) != tuple(q.shape) or not out.is_contiguous()
            or out.device != q.device):
        raise ValueError("out must be a contiguous float32 tensor of q's shape on q's device")


def dense_decode(K, V, lengths_dev, n_max, q, out=None, scratch=None, stream=None):
    """Full-scan exact attention.  q: bf16 [B, H_q, d] -> out f32 [B, H_q, d].  Over an e4m3
    cache (K a KV8 or PagedKV8; dense_decode8) `out` may also be bf16."""
    if isinstance(K, (KV8, PagedKV8)):
        return _cache_decode("dense_decode8", K, V, lengths_dev, n_max, q, None, out, scratch, stream)
    torch = _torch()
    B, H_kv = (q.shape[0], K.h_kv) if isinstance(K, PagedKV) else (K.shape[0], K.shape[1])
    H_q = q.shape[1]
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check_q_out(K, q, out)
    need = dense_scratch_bytes(B, H_kv, H_q, n_max)
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=q.device)
    kv = _kv(K, V)
    _check(lib().dense_decode(C.byref(kv), _ptr(lengths_dev), n_max, B, H_kv, H_q, 128, _ptr(q),
                              _ptr(out), _ptr(scratch), scratch.numel(), _stream(stream)),
           "dense_decode")
    return out


def dense_decode_noalloc(K, V, lengths_dev, n_max, q, out, stream=None):
    """dense_decode whose scratch is the library's static device array: no device memory
    is allocated by this call (the caller supplies `out`)."""
    if isinstance(K, (KV8, PagedKV8)):
        raise ValueError("dense_decode_noalloc reads bf16 caches")
    B, H_kv = (q.shape[0], K.h_kv) if isinstance(K, PagedKV) else (K.shape[0], K.shape[1])
    _check_q_out(K, q, out)
    kv = _kv(K, V)
    _check(lib().dense_decode_noalloc(C.byref(kv), _ptr(lengths_dev), n_max, B, H_kv, q.shape[1],
                                      128, _ptr(q), _ptr(out), _stream(stream)),
           "dense_decode_noalloc")
    return out


class _there:
    """The device `dev` made current, and work and allocations on `stream` (dev's current
    stream if None)."""

    def __init__(self, dev, stream):
        torch = _torch()
        if stream is not None and stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the cache on {dev}")
        self.cms = [torch.cuda.device(dev)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for cm in self.cms:
            cm.__enter__()

    def __exit__(self, *exc):
        for cm in reversed(self.cms):
            cm.__exit__(*exc)


def _here(dev, stream):
    """The cudaStream_t for work on `dev` if that is the current device and no stream is asked
    for; None if _there has to be entered first."""
    c = _torch()._C  # (torch.cuda's wrappers of these two cost 2 us a call)
    if stream is not None or dev.index != c._cuda_getDevice():
        return None
    return c._cuda_getCurrentRawStream(dev.index)


def _check_counts(t, B, dev, name):
    if t.dtype is not _torch().int32 or t.shape != (B,) or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous int32 tensor [{B}] on the cache's device")


@functools.lru_cache(maxsize=512)
def _scratch_bytes(entry, B, H_kv, H_q, n_max, dev_index) -> int:
    need = C.c_size_t(0)
    _check(getattr(lib(), entry + "_scratch_bytes")(B, H_kv, H_q, 128, n_max, C.byref(need)), entry)
    return need.value


def _cache_decode(entry, K, V, lengths_dev, n_max, q, diff, out, scratch, stream):
    torch = _torch()
    c, B, H_kv, positions, dev = _cache(K, V)
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return _cache_decode(entry, K, V, lengths_dev, n_max, q, diff, out, scratch, None)
    shape = q.shape
    if (q.dtype is not torch.bfloat16 or len(shape) != 3 or shape[0] != B or shape[2] != 128
            or not q.is_contiguous() or q.device != dev):
        raise ValueError("q must be a contiguous bf16 tensor [B, H_q, 128] on the cache's device")
    _check_counts(lengths_dev, B, dev, "lengths_dev")
    if not 1 <= n_max <= positions:
        raise ValueError(f"n_max must be between 1 and the cache's {positions} positions")
    H_q = shape[1]
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    elif (out.dtype not in (torch.float32, torch.bfloat16) or out.shape != shape or not out.is_contiguous()
          or out.device != dev):
        raise ValueError("out must be a contiguous float32 or bf16 tensor of q's shape on q's device")
    bf = out.dtype is torch.bfloat16
    own = None  # scratch of this call: from torch's allocator, given back to the stream's pool at the end
    if scratch is None:
        nbytes = _scratch_bytes(entry, B, H_kv, H_q, n_max, dev.index)
        if nbytes:  # (without the tensor around it, whose making costs 6 us between launches)
            own = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, s)
        at = own
    elif scratch.device != dev or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous tensor on the cache's device")
    else:
        nbytes = scratch.numel() * scratch.element_size()
        at = scratch.data_ptr()
    try:
        if diff is None:
            rc = lib().dense_decode8(C.byref(c), lengths_dev.data_ptr(), n_max, B, H_kv, H_q, 128, q.data_ptr(),
                                     out.data_ptr(), bf, at, nbytes, s)
        else:
            rc = lib().mog_diff_decode(C.byref(c), lengths_dev.data_ptr(), n_max, B, H_kv, H_q, 128, q.data_ptr(),
                                       C.byref(diff), out.data_ptr(), bf, at, nbytes, s)
    finally:
        if own is not None:
            torch._C._cuda_cudaCachingAllocator_raw_delete(own)
    if rc:
        _check(rc, entry)
    return out


def diff_decode(K, V, lengths_dev, n_max, q, lam, lambda_init, gamma=None, eps=1e-5, out=None, scratch=None,
                stream=None):
    """Differential decode attention (mog_diff_decode): a head is two halves of 64, q bf16
    [B, H_q, 128] = [q1 | q2] over keys [k1 | k2] and values of 128; the second softmax map is
    subtracted lambda times and the result normalised.  K, V: bf16 tensors, or K a PagedKV, KV8
    or PagedKV8.  lam: float32 [4, 64] or [H_q, 4, 64], the vectors l_q1, l_k1, l_q2, l_k2 of
    lambda = exp(l_q1.l_k1) - exp(l_q2.l_k2) + lambda_init; gamma: float32 [128] norm weights
    or None.  -> out f32 (or bf16 if given so) [B, H_q, 128]."""
    torch = _torch()
    shape, dev, shared = lam.shape, q.device, lam.dim() == 2
    if (lam.dtype is not torch.float32 or shape != ((4, 64) if shared else (q.shape[1], 4, 64))
            or not lam.is_contiguous() or lam.device != dev):
        raise ValueError("lam must be a contiguous float32 tensor [4, 64] or [H_q, 4, 64] on q's device")
    if gamma is not None and (gamma.dtype is not torch.float32 or gamma.shape != (128,) or not gamma.is_contiguous()
                              or gamma.device != dev):
        raise ValueError("gamma must be a contiguous float32 tensor [128] on q's device")
    d = DiffParams(lam.data_ptr(), None if gamma is None else gamma.data_ptr(), 1 if shared else shape[0], lambda_init,
                   eps)
    return _cache_decode("mog_diff_decode", K, V, lengths_dev, n_max, q, d, out, scratch, stream)


def diff_scratch_bytes(batch, h_kv, h_q, n_max) -> int:
    """Bytes of diff_decode's scratch on the current device."""
    return _scratch_bytes("mog_diff_decode", batch, h_kv, h_q, n_max, _torch().cuda.current_device()
                          if _torch().cuda.is_available() else -1)


def dense8_scratch_bytes(batch, h_kv, h_q, n_max) -> int:
    """Bytes of dense_decode's scratch over an e4m3 cache, on the current device."""
    return _scratch_bytes("dense_decode8", batch, h_kv, h_q, n_max, _torch().cuda.current_device()
                          if _torch().cuda.is_available() else -1)


def kv_store(K, V, pos, count, k_new, v_new, stream=None):
    """Write new rows into a cache (mog_kv_store): k_new, v_new bf16 [B, T, H_kv, 128] (any
    strides of whole 16-byte chunks, alike for both, last dim contiguous), token t < count[b] of
    sequence b to position pos[b] + t; pos, count int32 [B] on the device, count None for T
    each.  K, V: bf16 tensors [B, H_kv, n_cap, 128], or K a PagedKV, KV8 or PagedKV8 (rounded
    to e4m3 with a power-of-two scale per row)."""
    torch = _torch()
    c, B, H_kv, _, dev = _cache(K, V)
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return kv_store(K, V, pos, count, k_new, v_new)
    shape = k_new.shape
    if (len(shape) != 4 or k_new.dtype is not torch.bfloat16 or v_new.dtype is not torch.bfloat16
            or v_new.shape != shape or shape[0] != B or shape[2] != H_kv or shape[3] != 128 or k_new.device != dev
            or v_new.device != dev):
        raise ValueError(f"k_new and v_new must be bf16 tensors [{B}, T, {H_kv}, 128] on the cache's device")
    T = shape[1]

    def strides(t):  # 0 for a dim of one entry, whose stride does not count
        sb, st, sh, sd = t.stride()
        return sb if B > 1 else 0, st if T > 1 else 0, sh if H_kv > 1 else 0, sd

    sk = strides(k_new)
    if sk[3] != 1 or strides(v_new) != sk:
        raise ValueError("k_new and v_new must share strides, the last dim contiguous")
    _check_counts(pos, B, dev, "pos")
    at = None
    if count is not None:
        _check_counts(count, B, dev, "count")
        at = count.data_ptr()
    if T == 0:
        return
    rc = lib().mog_kv_store(C.byref(c), B, H_kv, 128, T, pos.data_ptr(), at, k_new.data_ptr(), v_new.data_ptr(), sk[0],
                            sk[1], sk[2], s)
    if rc:
        _check(rc, "mog_kv_store")


def _pool_desc(t):
    """mog_page_pool of a tensor whose first dim is the pages."""
    n, size = t.shape[0], t.element_size()
    page = t.numel() // n if n else 0
    if page == 0 or (n > 1 and t.stride(0) < page):
        raise ValueError("page pools must hold pages that do not overlap")
    return PagePoolDesc(t.data_ptr(), (t.stride(0) if n > 1 else page) * size, page * size)


class PagePool(_Fixed):
    """Sequences that share the pages of one or more paged caches (mog_pages): a block table
    [batch, pages_per_seq], the sequences' lengths and the pages' holders, all on the device.

    K, V: page pools [pages, H_kv, page_rows, 128] (heads_first) or [pages, page_rows, H_kv, 128],
    one tensor each or a list with one per layer, bf16, or float8_e4m3fn with k_scale, v_scale.  A page's
    elements must be contiguous.  block_table, lengths, refs: existing state, int32, used as it
    is; by default every sequence is empty.  The tensors are fixed once it is made; their contents may change between
    calls.  No method waits for the GPU but status()."""

    def __init__(self, K, V, batch, pages_per_seq, heads_first=True, k_scale=None, v_scale=None, block_table=None,
                 lengths=None, refs=None):
        torch = _torch()
        lists = [list(x) if isinstance(x, (list, tuple)) else [x] for x in (K, V)]
        self.K, self.V = lists
        if k_scale is not None or v_scale is not None:
            lists += [list(x) if isinstance(x, (list, tuple)) else [x] for x in (k_scale, v_scale)]
        self.k_scale, self.v_scale = lists[2:] if len(lists) == 4 else (None, None)
        if len({len(x) for x in lists}) != 1 or not self.K:
            raise ValueError("K, V and their scales must have one tensor per layer each")
        first = self.K[0]
        if first.dim() != 4 or first.shape[0] == 0:
            raise ValueError("page pools must have 4 dims and a page")
        self.device, n_pages = first.device, first.shape[0]
        self.heads_first, self.page_rows = heads_first, first.shape[2 if heads_first else 1]
        pools = [t for x in lists for t in x]
        rows = torch.float8_e4m3fn if len(lists) == 4 else torch.bfloat16
        if any(t.dtype != rows or t.dim() != 4 or t.shape != first.shape for t in self.K + self.V) or any(
                t.dtype != torch.float32 or t.dim() != 3 for x in lists[2:] for t in x):
            raise ValueError("K and V must be bf16 pools of one shape, or float8_e4m3fn with float32 k_scale and v_scale")
        for t in pools:
            if not t.is_cuda or t.device != self.device or t.shape[:3] != first.shape[:3] or not t[0].is_contiguous():
                raise ValueError("page pools must share a CUDA device and their first three dims, a page contiguous")
        for name, t, shape in (("block_table", block_table, (batch, pages_per_seq)), ("lengths", lengths, (batch,)),
                               ("refs", refs, (n_pages,))):
            if t is not None and (t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous()
                                  or t.device != self.device):
                raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on the pools' device")

        def state(t, shape, fill):
            return t if t is not None else torch.full(shape, fill, dtype=torch.int32, device=self.device)

        self.block_table = state(block_table, (batch, pages_per_seq), -1)
        self.lengths, self.refs = state(lengths, (batch,), 0), state(refs, (n_pages,), 0)
        need = C.c_size_t(0)
        _check(lib().mog_pages_work_bytes(n_pages, batch, C.byref(need)), "mog_pages_work_bytes")
        self.work = torch.zeros(need.value // 4, dtype=torch.int32, device=self.device)
        self._descs = (PagePoolDesc * len(pools))(*map(_pool_desc, pools))
        self._s = Pages(n_pages, self.page_rows, batch, pages_per_seq, self.block_table.data_ptr(),
                        self.lengths.data_ptr(), self.refs.data_ptr(), self.work.data_ptr(), need.value, self._descs,
                        len(pools))
        self.batch = batch
        self.pos, self.granted = torch.zeros_like(self.lengths), torch.zeros_like(self.lengths)
        self._lib, self._ref = lib(), C.byref(self._s)
        self._pos_ptr, self._granted_ptr = self.pos.data_ptr(), self.granted.data_ptr()
        self._layers = list(zip(*lists))  # what cache() hands out: the pools that the calls copy
        self._made = True

    def cache(self, layer=0):
        """The paged cache of a layer (PagedKV or PagedKV8), for the calls that take one."""
        return (PagedKV if self.k_scale is None else PagedKV8)(*self._layers[layer], self.block_table, self.page_rows,
                                                               self.heads_first)

    def _call(self, fn, stream, *args):
        s = _here(self.device, stream)
        if s is None:
            with _there(self.device, stream):
                return self._call(fn, None, *args)
        rc = fn(self._ref, *args, s)
        if rc:
            _check(rc, fn.__name__)

    def assign(self, src, stream=None):
        """Fork, reorder and free (mog_pages_assign): sequence b takes the pages and length that
        src[b] had (b: as it is; -1: none).  src: int32 [batch] on the device."""
        _check_counts(src, self.batch, self.device, "src")
        self._call(self._lib.mog_pages_assign, stream, src.data_ptr())

    def grow(self, n_new, stream=None):
        """Room for n_new[b] more tokens of every sequence (mog_pages_grow); a shared last page
        becomes private.  -> (self.pos, self.granted), int32 [batch]: where kv_store puts the new
        rows, and how many (0 everywhere if there was no room: see status()).  They are the
        same two tensors every time: the next grow overwrites them."""
        _check_counts(n_new, self.batch, self.device, "n_new")
        self._call(self._lib.mog_pages_grow, stream, n_new.data_ptr(), self._pos_ptr, self._granted_ptr)
        return self.pos, self.granted

    def compact(self, stream=None):
        """Move the pages in use to the front of the pools (mog_pages_compact)."""
        self._call(self._lib.mog_pages_compact, stream)

    def status(self, stream=None) -> int:
        """Wait for the stream, then read and clear the status of the calls so far: MOG_OK,
        MOG_ERR_CAPACITY (8) or MOG_ERR_DEVICE_CHECK (5)."""
        s = _here(self.device, stream)
        if s is None:
            with _there(self.device, stream):
                return self.status()
        return self._lib.mog_pages_status(self._ref, s)


def kmeans_assign(x, cent, stream=None, with_recheck=False):
    """One first-level assignment step: x bf16 [n, d] (row stride x.stride(0)), cent f32
    [k, d].  Returns (assign int32 [n], rows decided by the exact fallback), plus the rows
    the tensor-core pass left to the direct pass when with_recheck."""
    torch = _torch()
    n, k = x.shape[0], cent.shape[0]
    out = torch.empty(n, dtype=torch.int32, device=x.device)
    need = C.c_size_t(0)
    _check(lib().mog_kmeans_assign_scratch_bytes(n, k, 128, C.byref(need)), "scratch")
    scratch = torch.empty(need.value, dtype=torch.uint8, device=x.device)
    counts = (C.c_int32 * 2)()
    _check(lib().mog_kmeans_assign(_ptr(x), x.stride(0), n, _ptr(cent), k, 128, _ptr(out),
                                   _ptr(scratch), need.value, _stream(stream), counts),
           "mog_kmeans_assign")
    if with_recheck:
        return out, counts[0], counts[1]
    return out, counts[0]


def kmeans_assign_segments(x, rows, seg_off, cent, stream=None):
    """Second-level assignment step: segment s = rows[seg_off[s]:seg_off[s+1]] against
    cent[s] (f32 [n_seg, k, d])."""
    torch = _torch()
    out = torch.empty(rows.shape[0], dtype=torch.int32, device=x.device)
    n_seg, k = cent.shape[0], cent.shape[1]
    _check(lib().mog_kmeans_assign_segments(_ptr(x), x.stride(0), _ptr(rows), _ptr(seg_off), n_seg,
                                            _ptr(cent), k, 128, _ptr(out), _stream(stream)),
           "mog_kmeans_assign_segments")
    return out


def check_bounded_wait(limit, arrive, scratch, stream=None) -> int:
    """Run the library's bounded mbarrier wait on a barrier that is (arrive=True) or is not
    completed; returns the status code (MOG_OK or MOG_ERR_TIMEOUT = 6)."""
    return lib().mog_check_bounded_wait(limit, 1 if arrive else 0, _ptr(scratch), _stream(stream))
