"""Thin ctypes binding of libkvr (include/kvr.h): argument marshalling only.

Every step of the hot path runs in the library's CUDA kernels; this module
converts torch tensors to device pointers, host lists to C arrays, and
statuses to exceptions.  There is no fallback: if libkvr.so is missing the
import fails.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from operator import index
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvr.so")

KVR_OK = 0
KVR_DTYPE_BF16 = 0
KVR_DTYPE_FP32 = 1
KVR_SRC_LOCAL = 1 << 30
KVR_POSITIONS_COMPOSITE = 1
KVR_PREFILL_SKIP_PREFIX_CACHE = 2
KVR_WEIGHTS_ACCUMULATE = 1
KVR_EVICT_KEEP_ROTATION = 1
KVR_APPEND_TURNED = 1
KVR_POOL_KEYS_UNROTATED = 1
KVR_POOL_ROPE_INTERLEAVED = 2

STATUS = {0: "KVR_OK", 1: "KVR_ERR_INVALID_ARG", 2: "KVR_ERR_OUT_OF_RANGE", 3: "KVR_ERR_UNSUPPORTED",
          4: "KVR_ERR_CUDA", 5: "KVR_ERR_TIMEOUT", 6: "KVR_ERR_DEVICE_CHECK"}

EXPORTED = ("kvr_pool_register", "kvr_pool_unregister", "kvr_assemble", "kvr_query_attention",
            "kvr_prefill", "kvr_check", "kvr_status_string", "kvr_last_error", "kvr_attention_path",
            "kvr_set_timing_events", "kvr_selftest_wait", "kvr_assemble_noalloc", "kvr_pool_reserve",
            "kvr_shared_query_attention", "kvr_key_weights", "kvr_evict", "kvr_shared_path",
            "kvr_packed_page_bytes", "kvr_page_append", "kvr_page_attention", "kvr_page_pack", "kvr_page_unpack",
            "kvr_page_path")
PATH_UNBOUND, PATH_CUDA_CORES, PATH_TCGEN05 = -1, 0, 1
SHARED_NONE, SHARED_CUDA_CORES, SHARED_PARTS, SHARED_WHOLE = -1, 0, 1, 2
PAGE_NONE, PAGE_CUDA_CORES, PAGE_FEW, PAGE_MANY, PAGE_RESTORED, PAGE_JOINED = -1, 1, 2, 4, 8, 16


class KvrError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class PoolDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("n_entries", ctypes.c_int64), ("entry_len", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("stride", ctypes.c_int64 * 4), ("rope_theta", ctypes.c_double)]


class Span(ctypes.Structure):
    _fields_ = [("src", ctypes.c_int32), ("start", ctypes.c_int32), ("end", ctypes.c_int32)]


class LocalSrc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_int64),
                ("stride", ctypes.c_int64 * 3)]


class PageDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_rows", ctypes.c_int32), ("stride", ctypes.c_int64 * 3)]


class PackedDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libkvr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with rag_precomputed_kv_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.kvr_pool_register.argtypes = [ctypes.POINTER(PoolDesc), ctypes.POINTER(vp)]
    lib.kvr_pool_unregister.argtypes = [vp]
    lib.kvr_assemble.argtypes = [vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, ctypes.c_uint32, vp]
    lib.kvr_query_attention.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp]
    lib.kvr_prefill.argtypes = [vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, ctypes.c_uint32,
                                vp, vp, vp, vp, vp, ctypes.c_float, vp]
    lib.kvr_shared_query_attention.argtypes = [vp, i32] + [vp] * 14 + [ctypes.c_float, vp]
    lib.kvr_key_weights.argtypes = [vp, i32] + [vp] * 6 + [ctypes.c_float, ctypes.c_uint32, vp]
    lib.kvr_evict.argtypes = [vp, i32, vp, vp, vp, i32, i32] + [vp] * 8 + [ctypes.c_uint32, vp]
    lib.kvr_packed_page_bytes.argtypes = [vp, i32]
    lib.kvr_packed_page_bytes.restype = i64
    lib.kvr_page_append.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, ctypes.c_uint32, vp]
    lib.kvr_page_attention.argtypes = [vp, vp, i32, vp, i32] + [vp] * 5 + [i32, i32, vp, vp, i32, vp, ctypes.c_float, vp]
    lib.kvr_page_pack.argtypes = [vp, vp, i32, vp, i32, vp, vp, i32, vp, vp, vp]
    lib.kvr_page_unpack.argtypes = [vp, vp, i32, vp, i32, vp, vp, i32, vp, vp, vp]
    lib.kvr_check.argtypes = [vp, vp]
    lib.kvr_assemble_noalloc.argtypes = [ctypes.POINTER(PoolDesc), i32, vp, vp, vp, i32, vp, vp, vp, vp, vp,
                                         vp, ctypes.c_uint32, vp]
    lib.kvr_selftest_wait.argtypes = [vp, ctypes.c_uint64, vp]
    lib.kvr_pool_reserve.argtypes = [vp, i32, i32, i32, i64]
    lib.kvr_status_string.restype = ctypes.c_char_p
    lib.kvr_status_string.argtypes = [ctypes.c_int]
    lib.kvr_last_error.restype = ctypes.c_char_p
    lib.kvr_set_timing_events.argtypes = [vp, vp]
    lib.kvr_set_timing_events.restype = ctypes.c_int
    lib.kvr_attention_path.argtypes = [vp]
    lib.kvr_attention_path.restype = ctypes.c_int32
    lib.kvr_shared_path.argtypes = [vp]
    lib.kvr_shared_path.restype = ctypes.c_int32
    lib.kvr_page_path.argtypes = [vp]
    lib.kvr_page_path.restype = ctypes.c_int32
    for name in ("kvr_pool_register", "kvr_pool_unregister", "kvr_assemble", "kvr_query_attention",
                 "kvr_prefill", "kvr_check", "kvr_selftest_wait", "kvr_assemble_noalloc", "kvr_pool_reserve",
                 "kvr_shared_query_attention", "kvr_key_weights", "kvr_evict", "kvr_page_append", "kvr_page_attention",
                 "kvr_page_pack", "kvr_page_unpack"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _raise(st: int):
    if st != KVR_OK:
        raise KvrError(st, load().kvr_last_error().decode())


_raw_stream = None   # () -> the current stream's handle, once CUDA is initialised


def _stream_ptr(stream) -> Optional[int]:
    global _raw_stream
    if stream is None:
        if _raw_stream is not None:   # 3 us less than a Stream object
            return _raw_stream()
        import torch
        raw, dev = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if raw is not None and dev is not None and torch.cuda.is_initialized():
            _raw_stream = lambda: raw(dev())
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _i64(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64))


def _ints(name: str, a, code: str, n: Optional[int] = None):
    """``a`` as a C array of int32 ("i") or int64 ("q"): (keep-alive, address,
    length); ``n``: the length it must have.  Lists take the short way, which
    costs a tenth of numpy's."""
    if isinstance(a, (list, tuple)):
        c = array(code, a)
        addr, m = c.buffer_info()
    else:
        a = np.asarray(a)
        c = np.ascontiguousarray(a, dtype=np.int32 if code == "i" else np.int64)
        if c.ndim != 1:
            raise ValueError(f"{name} must be one-dimensional, got shape {c.shape}")
        if a.dtype != c.dtype and a.size and (a.dtype.kind not in "iu" or (a != c).any()):
            raise ValueError(f"{name} must hold {8 * c.itemsize}-bit integers")
        addr, m = c.ctypes.data, len(c)
    if n is not None and m != n:
        raise ValueError(f"{name} must hold {n} values, got {m}")
    return c, addr, m


def _shared_tables(go, po, pl, co, ol, qo):
    """`_ints` of a shared-prefix call's six tables: (keep-alive, groups, query
    tokens, rows of the caches, rows of the prefix or 0, the six addresses).  Lists
    of the right lengths go into one C array of either type (half the time of six)."""
    if type(go) is type(po) is type(pl) is type(co) is type(ol) is type(qo) is list and go:
        n, b = len(go), go[-1]
        if len(pl) == n - 1 and len(po) == n and len(ol) == b and len(qo) == len(co) == b + 1:
            c32, c64 = array("i", go + pl + ol + qo), array("q", po + co)
            a32, a64 = c32.buffer_info()[0], c64.buffer_info()[0]
            own = a32 + 8 * n - 4
            return (c32, c64), n - 1, qo[-1], co[-1], po[-1] if any(pl) else 0, a32, a64, a32 + 4 * n, a64 + 8 * n, own, own + 4 * b
    g = _ints("group_offsets", go, "i")
    if g[2] == 0:
        raise ValueError("group_offsets must hold at least one value")
    n, b = g[2] - 1, max(0, int(g[0][-1]))   # (the library refuses a negative one)
    t = (g, _ints("prefix_offsets", po, "q", n + 1), _ints("prefix_len", pl, "i", n), _ints("cache_offsets", co, "q", b + 1),
         _ints("own_len", ol, "i", b), _ints("q_offsets", qo, "i", b + 1))
    return (t, n, int(t[5][0][-1]), int(t[3][0][-1]), int(t[1][0][-1]) if any(t[2][0]) else 0, *(x[1] for x in t))


def _data(name: str, t, dtype, n: int) -> Optional[int]:
    """The address of a tensor that a call reads or writes as ``n`` elements of
    ``dtype`` one behind the other (None: NULL, which the library judges)."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.is_contiguous() and t.numel() >= n and (t.is_cuda or t.is_pinned())):
        if t.dtype is not dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor")
        if t.numel() < n:
            raise ValueError(f"{name} must hold at least {n} values, got {t.numel()}")
        raise ValueError(f"{name} must be in device or pinned host memory")
    return t.data_ptr()


def _int32(name: str, x) -> int:
    """``x``, an integer that fits 32 bits."""
    i = index(x)
    if not -(1 << 31) <= i < 1 << 31:
        raise ValueError(f"{name} must be a 32-bit integer, got {i}")
    return i


def _page_table(name: str, a, batch: int):
    """``a`` as a C array of int32 [batch][width]: (keep-alive, address, width)."""
    if a is None:
        return None, None, 0
    if hasattr(a, "is_cuda"):
        if a.is_cuda:
            raise ValueError(f"{name} must be in host memory")
        import torch
        shape = a.shape
        if a.dtype is torch.int32 and len(shape) == 2 and shape[0] == batch and a.is_contiguous():
            return a, a.data_ptr(), shape[1]
        a = a.numpy()
    elif not isinstance(a, np.ndarray):
        a = [list(r) for r in a]
        width = max(map(len, a), default=0)
        a = np.array(array("i", [x for r in a for x in r + [-1] * (width - len(r))]), np.int32).reshape(len(a), width)
    c = np.ascontiguousarray(a, dtype=np.int32)
    if c.ndim != 2 or c.shape[0] != batch:
        raise ValueError(f"{name} must be [{batch}, pages], got shape {c.shape}")
    if a.dtype != c.dtype and a.size and (a.dtype.kind not in "iu" or (a != c).any()):
        raise ValueError(f"{name} must hold 32-bit integers")
    return c, c.ctypes.data, c.shape[1]


class Pages:
    """The pages of a cache: ``k``, ``v`` ``[n_pages, layers, kv_heads, page_rows,
    head_dim]``, of equal strides, whose rows are one behind the other (kvr_pages).
    The tensors must outlive the calls that use them."""

    def __init__(self, k, v):
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype is not v.dtype:
            raise ValueError("k and v must be alike, [n_pages, layers, kv_heads, page_rows, head_dim]")
        if k.stride(4) != 1 or (k.shape[3] > 1 and k.stride(3) != k.shape[4]):
            raise ValueError("the rows of a page must be contiguous")
        if not (k.is_cuda and v.is_cuda):
            raise ValueError("pages must be in device memory")
        self.k, self.v = k, v
        self.page_rows, self.shape, self.dtype = k.shape[3], (k.shape[1], k.shape[2], k.shape[4]), k.dtype
        self._d = PageDesc(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[3], (ctypes.c_int64 * 3)(*k.stride()[:3]))
        self._p = ctypes.addressof(self._d)


class PackedPages:
    """Packed pages: ``data`` ``[n_pages, bytes]`` (uint8), ``bytes`` those of
    :meth:`Pool.packed_page_bytes` for ``page_rows`` (kvr_packed_pages)."""

    def __init__(self, data, page_rows: int):
        import torch
        if data.dtype is not torch.uint8 or data.dim() != 2 or not data.is_contiguous() or not data.is_cuda:
            raise ValueError("data must be a contiguous uint8 device tensor [n_pages, bytes]")
        self.data, self.page_rows = data, _int32("page_rows", page_rows)
        self._d = PackedDesc(data.data_ptr(), data.shape[0])
        self._p = ctypes.addressof(self._d)


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data


def _span_args(span_offsets, spans, cache_offsets, locals_):
    so = _i32(span_offsets)
    sp = _i32(spans).reshape(-1, 3)
    co = _i64(cache_offsets)
    loc = (LocalSrc * max(1, len(locals_)))()
    for i, (lk, lv) in enumerate(locals_):
        assert lk.stride() == lv.stride() and lk.stride(-1) == 1
        loc[i] = LocalSrc(_ptr(lk), _ptr(lv), lk.shape[2], (ctypes.c_int64 * 3)(*lk.stride()[:3]))
    return so, sp, co, loc, len(so) - 1


def _pool_desc(k, v, n_q_heads: int, rope_theta: float, keys_unrotated: bool, rope_interleaved: bool):
    import torch
    assert k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype
    assert k.stride(-1) == 1
    dt = {torch.bfloat16: KVR_DTYPE_BF16, torch.float32: KVR_DTYPE_FP32}[k.dtype]
    E, L, H, T, D = k.shape
    flags = ((KVR_POOL_KEYS_UNROTATED if keys_unrotated else 0)
             | (KVR_POOL_ROPE_INTERLEAVED if rope_interleaved else 0))
    return PoolDesc(L, n_q_heads, H, D, dt, flags, E, T, _ptr(k), _ptr(v),
                    (ctypes.c_int64 * 4)(*k.stride()[:4]), float(rope_theta))


def assemble_noalloc(k, v, n_q_heads: int, rope_theta: float, span_offsets: Sequence[int], spans,
                     cache_offsets, cache_k, cache_v, locals_=(), pos_ids=None, src_map=None,
                     composite: bool = False, keys_unrotated: bool = False,
                     rope_interleaved: bool = False, stream=None) -> np.ndarray:
    """kvr_assemble_noalloc: kvr_assemble for callers that cannot allocate.

    No pool handle: the pool tensors ``k``, ``v`` are described as for
    :class:`Pool` on every call.  Returns the per-request prefix lengths
    (numpy int32).  The library's fixed scratch is shared by all such calls
    (see the header for its limits and its one-call-at-a-time rule).
    """
    d = _pool_desc(k, v, n_q_heads, rope_theta, keys_unrotated, rope_interleaved)
    so, sp, co, loc, batch = _span_args(span_offsets, spans, cache_offsets, locals_)
    plen = np.zeros(max(batch, 1), np.int32)
    _raise(load().kvr_assemble_noalloc(ctypes.byref(d), batch, _np_ptr(so), _np_ptr(sp) if sp.size else None,
                                       ctypes.cast(loc, ctypes.c_void_p) if len(locals_) else None,
                                       len(locals_), _np_ptr(co), _ptr(cache_k), _ptr(cache_v),
                                       _ptr(pos_ids), _ptr(src_map), _np_ptr(plen),
                                       KVR_POSITIONS_COMPOSITE if composite else 0, _stream_ptr(stream)))
    return plen[:batch]


class Pool:
    """A registered pool of precomputed chunk caches.

    ``k``, ``v``: tensors ``[entries, layers, kv_heads, entry_len, head_dim]`` in
    device memory or pinned host memory (any strides with head_dim contiguous),
    keys rotated at entry-local positions (or, with ``keys_unrotated``, before
    RoPE).  ``rope_interleaved``:
    RoPE pairs are (x_2i, x_2i+1) instead of (x_i, x_i+D/2), for the stored
    keys and every rotation the library makes.  The tensors must outlive the
    pool.
    """

    def __init__(self, k, v, n_q_heads: int, rope_theta: float, keys_unrotated: bool = False,
                 rope_interleaved: bool = False):
        lib = load()
        d = _pool_desc(k, v, n_q_heads, rope_theta, keys_unrotated, rope_interleaved)
        _, L, H, _, D = k.shape
        h = ctypes.c_void_p()
        _raise(lib.kvr_pool_register(ctypes.byref(d), ctypes.byref(h)))
        self._h = h
        self._keep = (k, v)
        self.n_layers, self.n_kv_heads, self.n_q_heads, self.head_dim = L, H, n_q_heads, D
        self.dtype = k.dtype
        self._layout = (L, H, D)
        # elements of a cache row in every layer and kv head, and of a token's queries in a layer
        self._row, self._heads, self._wide = L * H * D, H * D, n_q_heads * D

    def reserve(self, max_batch: int = 0, max_spans: int = 0, max_locals: int = 0, max_query_tokens: int = 0):
        """kvr_pool_reserve: bind the pool to the current device and allocate
        now every staging and scratch buffer that calls within these limits
        need; later calls within them never allocate."""
        _raise(load().kvr_pool_reserve(self._h, int(max_batch), int(max_spans), int(max_locals),
                                       int(max_query_tokens)))

    def close(self):
        if getattr(self, "_h", None):
            load().kvr_pool_unregister(self._h)
            self._h = None

    __del__ = close

    def assemble(self, span_offsets: Sequence[int], spans, cache_offsets, cache_k, cache_v,
                 locals_=(), pos_ids=None, src_map=None, composite: bool = False, stream=None):
        """kvr_assemble; returns the per-request prefix lengths (numpy int32)."""
        so, sp, co, loc, batch = _span_args(span_offsets, spans, cache_offsets, locals_)
        plen = np.zeros(max(batch, 1), np.int32)
        _raise(load().kvr_assemble(self._h, batch, _np_ptr(so), _np_ptr(sp) if sp.size else None,
                                   ctypes.cast(loc, ctypes.c_void_p) if len(locals_) else None,
                                   len(locals_), _np_ptr(co),
                                   _ptr(cache_k), _ptr(cache_v), _ptr(pos_ids), _ptr(src_map),
                                   _np_ptr(plen), KVR_POSITIONS_COMPOSITE if composite else 0,
                                   _stream_ptr(stream)))
        return plen[:batch]

    def prefill(self, span_offsets: Sequence[int], spans, cache_offsets, cache_k, cache_v,
                q_offsets, q, kq, vq, out, locals_=(), pos_ids=None, src_map=None,
                composite: bool = False, softmax_scale: float = 0.0, skip_prefix_cache: bool = False,
                stream=None):
        """kvr_prefill (assemble + query attention in one call); returns the
        per-request prefix lengths (numpy int32).  skip_prefix_cache: the
        attention gathers the prefix from the pool and the cache's prefix rows
        are not written (KVR_PREFILL_SKIP_PREFIX_CACHE)."""
        so, sp, co, loc, batch = _span_args(span_offsets, spans, cache_offsets, locals_)
        qo = _i32(q_offsets)
        plen = np.zeros(max(batch, 1), np.int32)
        _raise(load().kvr_prefill(self._h, batch, _np_ptr(so), _np_ptr(sp) if sp.size else None,
                                  ctypes.cast(loc, ctypes.c_void_p) if len(locals_) else None,
                                  len(locals_), _np_ptr(co),
                                  _ptr(cache_k), _ptr(cache_v), _ptr(pos_ids), _ptr(src_map),
                                  _np_ptr(plen), (KVR_POSITIONS_COMPOSITE if composite else 0) |
                                  (KVR_PREFILL_SKIP_PREFIX_CACHE if skip_prefix_cache else 0),
                                  _np_ptr(qo), _ptr(q), _ptr(kq), _ptr(vq), _ptr(out),
                                  float(softmax_scale), _stream_ptr(stream)))
        return plen[:batch]

    def query_attention(self, cache_offsets, prefix_len, q_offsets, q, kq, vq, cache_k, cache_v,
                        out, softmax_scale: float = 0.0, stream=None):
        """kvr_query_attention (appends the query K/V to the cache, writes out).
        ``q``, ``kq``, ``vq`` and ``out`` may be device or pinned host tensors;
        with one token per request the call is a decode step (one kernel)."""
        co, pl, qo = _i64(cache_offsets), _i32(prefix_len), _i32(q_offsets)
        _raise(load().kvr_query_attention(self._h, len(qo) - 1, _np_ptr(co), _np_ptr(pl), _np_ptr(qo),
                                          _ptr(q), _ptr(kq), _ptr(vq), _ptr(cache_k), _ptr(cache_v),
                                          _ptr(out), float(softmax_scale), _stream_ptr(stream)))

    def shared_query_attention(self, group_offsets, prefix_offsets, prefix_len, prefix_k, prefix_v, cache_offsets,
                               own_len, q_offsets, q, kq, vq, cache_k, cache_v, out, softmax_scale: float = 0.0,
                               stream=None):
        """kvr_shared_query_attention: query attention of groups of requests,
        each over its group's shared prefix block (``prefix_k``, ``prefix_v``,
        read only) and the requests' own rows, to which the query K/V are
        appended; writes ``out``."""
        keep, n, tokens, rows, pre, go, po, pl, co, ol, qo = _shared_tables(group_offsets, prefix_offsets, prefix_len,
                                                                            cache_offsets, own_len, q_offsets)
        if tokens <= 0:   # nothing to do, or refused
            ptrs = map(_ptr, (prefix_k, prefix_v, q, kq, vq, cache_k, cache_v, out))
        else:
            d, wide, heads = self.dtype, self._wide * self.n_layers * tokens, self._heads * self.n_layers * tokens
            rows, pre = self._row * rows, self._row * pre
            ptrs = (_data("prefix_k", prefix_k, d, pre), _data("prefix_v", prefix_v, d, pre), _data("q", q, d, wide),
                    _data("kq", kq, d, heads), _data("vq", vq, d, heads), _data("cache_k", cache_k, d, rows),
                    _data("cache_v", cache_v, d, rows), _data("out", out, d, wide))
        pk, pv, q_, kq_, vq_, ck, cv, out_ = ptrs
        _raise(load().kvr_shared_query_attention(self._h, n, go, po, pl, pk, pv, co, ol, qo, q_, kq_, vq_, ck, cv, out_,
                                                 float(softmax_scale), _stream_ptr(stream)))

    def key_weights(self, cache_offsets, prefix_len, q_offsets, q, cache_k, weights, softmax_scale: float = 0.0,
                    accumulate: bool = False, stream=None):
        """kvr_key_weights: the attention weight each cached key receives from
        the query tokens (fp32, one value per cache row), written to
        ``weights`` or, with ``accumulate``, added to it."""
        import torch
        qo = _ints("q_offsets", q_offsets, "i")
        n = qo[2] - 1
        co, pl = _ints("cache_offsets", cache_offsets, "q", n + 1), _ints("prefix_len", prefix_len, "i", n)
        rows, tokens = (int(co[0][-1]), int(qo[0][-1])) if n >= 0 else (0, 0)
        w = _data("weights", weights, torch.float32, self.n_layers * self.n_kv_heads * rows)
        ck = _data("cache_k", cache_k, self.dtype, self._row * rows)
        q_ = _data("q", q, self.dtype, self.n_layers * tokens * self._wide)
        _raise(load().kvr_key_weights(self._h, n, co[1], pl[1], qo[1], q_, ck, w, float(softmax_scale),
                                      KVR_WEIGHTS_ACCUMULATE if accumulate else 0, _stream_ptr(stream)))

    def evict(self, cache_offsets, kv_len, keep, weights, cache_k, cache_v, kept, dst_offsets=None, dst_k=None,
              dst_v=None, dst_weights=None, n_first: int = 0, n_recent: int = 0, keep_rotation: bool = False,
              stream=None):
        """kvr_evict: keep the ``keep[b]`` heaviest rows of each block (the
        first ``n_first`` and last ``n_recent`` always), moved to rows 0.. with
        their keys turned to the new positions; ``kept`` (int32) receives the
        rows.  Without ``dst_k`` the cache and the weights are evicted in
        place.  Returns the rows each request holds afterwards (numpy int32)."""
        import torch
        if dst_k is None:
            if dst_v is not None or dst_weights is not None or dst_offsets is not None:
                raise ValueError("dst_offsets, dst_v and dst_weights go with dst_k")
            dst_offsets, dst_k, dst_v, dst_weights = cache_offsets, cache_k, cache_v, weights
        elif dst_offsets is None:
            raise ValueError("dst_k needs dst_offsets")
        kl = _ints("kv_len", kv_len, "i")
        n = kl[2]
        kp, co = _ints("keep", keep, "i", n), _ints("cache_offsets", cache_offsets, "q", n + 1)
        do = _ints("dst_offsets", dst_offsets, "q", n + 1)
        units, d, rows, d_rows = self.n_layers * self.n_kv_heads, self.dtype, int(co[0][-1]), int(do[0][-1])
        kept_ = _data("kept", kept, torch.int32, units * sum(map(min, kl[0].tolist(), kp[0].tolist())))
        w, dw = _data("weights", weights, torch.float32, units * rows), _data("dst_weights", dst_weights, torch.float32, units * d_rows)
        ck, cv = _data("cache_k", cache_k, d, self._row * rows), _data("cache_v", cache_v, d, self._row * rows)
        dk, dv = _data("dst_k", dst_k, d, self._row * d_rows), _data("dst_v", dst_v, d, self._row * d_rows)
        _raise(load().kvr_evict(self._h, n, co[1], kl[1], kp[1], int(n_first), int(n_recent), w, ck, cv, do[1], dk, dv, dw,
                                kept_, KVR_EVICT_KEEP_ROTATION if keep_rotation else 0, _stream_ptr(stream)))
        return np.minimum(kl[0], kp[0], dtype=np.int32)

    def _pages(self, pages: "Pages") -> int:
        if pages.shape != self._layout or pages.dtype is not self.dtype:
            raise ValueError(f"pages of {pages.shape} (layers, kv heads, head dim), {pages.dtype} do not fit the pool")
        return pages._p

    def _packed(self, packed: "PackedPages", pages: "Pages") -> int:
        if packed.page_rows != pages.page_rows:
            raise ValueError(f"packed pages of {packed.page_rows} rows, pages of {pages.page_rows}")
        n = self.packed_page_bytes(packed.page_rows)
        if n and packed.data.shape[1] != n:   # (n 0: the library refuses the call)
            raise ValueError(f"packed pages must have {n} bytes, got {packed.data.shape[1]}")
        return packed._p

    def packed_page_bytes(self, page_rows: int) -> int:
        """kvr_packed_page_bytes: 0 where the pool's rows cannot be packed."""
        return int(load().kvr_packed_page_bytes(self._h, _int32("page_rows", page_rows)))

    def packed_pages(self, n_pages: int, page_rows: int) -> "PackedPages":
        """New packed pages (zeros: scales of 0) on the current device."""
        import torch
        n = self.packed_page_bytes(page_rows)
        if n == 0:
            raise ValueError("packed pages need a bf16 pool with head_dim 128 and page_rows a multiple of 32")
        return PackedPages(torch.zeros((n_pages, n), dtype=torch.uint8, device="cuda"), page_rows)

    def page_append(self, pages: "Pages", table, start, q_offsets, k, v, turned: bool = False, stream=None):
        """kvr_page_append: token t of request b becomes row ``start[b] + t`` of
        its pages (``table`` ``[batch, width]``, host memory), its key turned to
        that position or, with ``turned``, copied.  ``k``, ``v``: ``[layers, T,
        kv_heads, head_dim]``, of equal strides (a stitched block seen token by
        token: ``block.view(L, H, R, D).transpose(1, 2)``)."""
        qo = _ints("q_offsets", q_offsets, "i")
        n = qo[2] - 1
        st, tab, p = _ints("start", start, "i", n), _page_table("table", table, n), self._pages(pages)
        tokens = int(qo[0][-1]) if n >= 0 else 0
        d, s3, shape = self.dtype, k.stride(), k.shape
        if not (k.dtype is d and v.dtype is d and k.is_cuda and v.is_cuda and v.stride() == s3 and v.shape == shape):
            raise ValueError("k and v must be alike, device tensors [layers, T, kv_heads, head_dim] of the pool's type and of equal strides")
        if len(shape) != 4 or shape[0] != self.n_layers or shape[1] < tokens or shape[2] != self.n_kv_heads or shape[3] != self.head_dim:
            raise ValueError(f"k and v must hold {tokens} tokens of the pool's layout, got {tuple(shape)}")
        if s3[3] != 1:
            raise ValueError("the rows of k and v must be contiguous")
        strides = array("q", s3)
        _raise(load().kvr_page_append(self._h, p, n, tab[1], tab[2], st[1], qo[1], k.data_ptr(), v.data_ptr(),
                                      strides.buffer_info()[0], KVR_APPEND_TURNED if turned else 0, _stream_ptr(stream)))

    def page_attention(self, pages: "Pages", table, kv_len, q_offsets, q, out, q_pos=None, window: int = 0,
                       n_first: int = 0, packed: Optional["PackedPages"] = None, packed_table=None, packed_len=None,
                       softmax_scale: float = 0.0, stream=None):
        """kvr_page_attention: attention of ``q`` ``[layers, T, q_heads, head_dim]``
        (T: ``q_offsets[-1]``) over the paged cache, written to ``out``; with
        ``window``, over the last ``window`` rows before each query and the first
        ``n_first``.  ``packed``: rows below ``packed_len[b]`` are read from these
        packed pages, through ``packed_table``."""
        qo = _ints("q_offsets", q_offsets, "i")
        n = qo[2] - 1
        kl, tab, p = _ints("kv_len", kv_len, "i", n), _page_table("table", table, n), self._pages(pages)
        qp = (None, None) if q_pos is None else _ints("q_pos", q_pos, "i", n)
        pk, ptab, pl = None, (None, None, 0), (None, None)
        if packed is not None:
            if packed_len is None:
                raise ValueError("packed goes with packed_table and packed_len")
            pk, ptab, pl = self._packed(packed, pages), _page_table("packed_table", packed_table, n), _ints("packed_len", packed_len, "i", n)
        elif packed_table is not None or packed_len is not None:
            raise ValueError("packed_table and packed_len go with packed")
        tokens = int(qo[0][-1]) if n >= 0 else 0
        size = self.n_layers * tokens * self._wide
        for name, x in (("q", q), ("out", out)):   # (the layers lie as many tokens apart as there are)
            if x is not None and self.n_layers > 1 and x.dim() == 4 and x.shape[0] == self.n_layers and x.shape[1] != tokens:
                raise ValueError(f"{name} must hold {tokens} tokens in each layer, got {x.shape[1]}")
        for name, x in (("q", q), ("out", out)):
            if x is not None and not x.is_cuda:
                raise ValueError(f"{name} must be in device memory")
        q_, o_ = _data("q", q, self.dtype, size), _data("out", out, self.dtype, size)
        _raise(load().kvr_page_attention(self._h, p, n, tab[1], tab[2], kl[1], qp[1], qo[1], q_, o_,
                                         _int32("window", window), _int32("n_first", n_first), pk, ptab[1], ptab[2], pl[1],
                                         float(softmax_scale), _stream_ptr(stream)))

    def page_pack(self, pages: "Pages", table, packed: "PackedPages", packed_table, begin, end, stream=None):
        """kvr_page_pack: rows ``begin[b]`` .. ``end[b] - 1`` (multiples of 32) of
        each request's pages into its packed pages."""
        b = _ints("begin", begin, "i")
        e, t, pt = _ints("end", end, "i", b[2]), _page_table("table", table, b[2]), _page_table("packed_table", packed_table, b[2])
        _raise(load().kvr_page_pack(self._h, self._pages(pages), b[2], t[1], t[2], self._packed(packed, pages), pt[1], pt[2],
                                    b[1], e[1], _stream_ptr(stream)))

    def page_unpack(self, packed: "PackedPages", packed_table, pages: "Pages", table, begin, end, stream=None):
        """kvr_page_unpack: the other way, rounded to bf16."""
        b = _ints("begin", begin, "i")
        e, t, pt = _ints("end", end, "i", b[2]), _page_table("table", table, b[2]), _page_table("packed_table", packed_table, b[2])
        _raise(load().kvr_page_unpack(self._h, self._packed(packed, pages), b[2], pt[1], pt[2], self._pages(pages), t[1], t[2],
                                      b[1], e[1], _stream_ptr(stream)))

    @property
    def attention_path(self) -> int:
        """PATH_TCGEN05, PATH_CUDA_CORES, or PATH_UNBOUND before the first call."""
        return int(load().kvr_attention_path(self._h))

    @property
    def shared_path(self) -> int:
        """Kernels of the last :meth:`shared_query_attention` that enqueued work:
        SHARED_CUDA_CORES, SHARED_PARTS, SHARED_WHOLE, or SHARED_NONE before it."""
        return int(load().kvr_shared_path(self._h))

    @property
    def page_path(self) -> int:
        """Kernels of the last :meth:`page_attention` that enqueued work: PAGE_ bits, and 256
        times the launches that many query rows took; or PAGE_NONE before it."""
        return int(load().kvr_page_path(self._h))

    def set_timing_events(self, events):
        """Six torch.cuda.Event(enable_timing=True) recorded around the
        assemble, query-append and attention kernels (None turns it off)."""
        if events is None:
            _raise(load().kvr_set_timing_events(self._h, None))
            return
        arr = (ctypes.c_void_p * 6)(*[int(e.cuda_event) for e in events])
        _raise(load().kvr_set_timing_events(self._h, ctypes.cast(arr, ctypes.c_void_p)))

    def selftest_wait(self, limit_ns: int, stream=None):
        """Enqueue a kernel whose bounded wait runs out after ``limit_ns``
        (the library's timeout path); the next :meth:`check` raises
        KVR_ERR_TIMEOUT."""
        _raise(load().kvr_selftest_wait(self._h, int(limit_ns), _stream_ptr(stream)))

    def check(self, stream=None):
        """kvr_check: synchronize and raise on a device-recorded error."""
        _raise(load().kvr_check(self._h, _stream_ptr(stream)))
