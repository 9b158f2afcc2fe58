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
KVR_POOL_KEYS_UNROTATED = 1
KVR_POOL_ROPE_INTERLEAVED = 2

STATUS = {0: "KVR_OK", 1: "KVR_ERR_INVALID_ARG", 2: "KVR_ERR_OUT_OF_RANGE", 3: "KVR_ERR_UNSUPPORTED",
          4: "KVR_ERR_CUDA", 5: "KVR_ERR_TIMEOUT", 6: "KVR_ERR_DEVICE_CHECK"}

EXPORTED = ("kvr_pool_register", "kvr_pool_unregister", "kvr_assemble", "kvr_query_attention",
            "kvr_prefill", "kvr_check", "kvr_status_string", "kvr_last_error", "kvr_attention_path",
            "kvr_set_timing_events", "kvr_selftest_wait", "kvr_assemble_noalloc", "kvr_pool_reserve",
            "kvr_shared_query_attention", "kvr_key_weights", "kvr_evict", "kvr_shared_path")
PATH_UNBOUND, PATH_CUDA_CORES, PATH_TCGEN05 = -1, 0, 1
SHARED_NONE, SHARED_CUDA_CORES, SHARED_PARTS, SHARED_WHOLE = -1, 0, 1, 2


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
    for name in ("kvr_pool_register", "kvr_pool_unregister", "kvr_assemble", "kvr_query_attention",
                 "kvr_prefill", "kvr_check", "kvr_selftest_wait", "kvr_assemble_noalloc", "kvr_pool_reserve",
                 "kvr_shared_query_attention", "kvr_key_weights", "kvr_evict"):
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

    @property
    def attention_path(self) -> int:
        """PATH_TCGEN05, PATH_CUDA_CORES, or PATH_UNBOUND before the first call."""
        return int(load().kvr_attention_path(self._h))

    @property
    def shared_path(self) -> int:
        """Kernels of the last :meth:`shared_query_attention` that enqueued work:
        SHARED_CUDA_CORES, SHARED_PARTS, SHARED_WHOLE, or SHARED_NONE before it."""
        return int(load().kvr_shared_path(self._h))

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
