"""Shared-prefix attention, key weights and eviction on the CPU: every refused
argument is refused with a status, before any GPU work."""
import ctypes

import numpy as np
import pytest

from rag_precomputed_kv_gb300 import build as B

A, Bp, C, Dp, E, F = (0x10000000 * (i + 1) for i in range(6))   # far apart, aligned


@pytest.fixture(scope="module")
def lib():
    B.build()
    from rag_precomputed_kv_gb300 import kvr
    return kvr.load()


@pytest.fixture(scope="module")
def pool(lib):
    from rag_precomputed_kv_gb300 import kvr
    d = kvr.PoolDesc(2, 8, 2, 128, kvr.KVR_DTYPE_BF16, 0, 4, 512, 0x10000, 0x20000,
                     (ctypes.c_int64 * 4)(2 * 2 * 512 * 128, 2 * 512 * 128, 512 * 128, 128), 1e6)
    h = ctypes.c_void_p()
    assert lib.kvr_pool_register(ctypes.byref(d), ctypes.byref(h)) == 0
    yield h
    lib.kvr_pool_unregister(h)


def _p(x, dt):
    if x is None:
        return None, None
    a = np.ascontiguousarray(x, dt)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def shared(lib, h, go=(0, 2), po=(0, 100), pl=(90,), co=(0, 20, 40), own=(3, 4), qo=(0, 1, 2), pk=A, pv=Bp, q=C, kq=C,
           vq=C, ck=Dp, cv=E, out=F, scale=0.0, n=None):
    keep = [_p(go, np.int32), _p(po, np.int64), _p(pl, np.int32), _p(co, np.int64), _p(own, np.int32), _p(qo, np.int32)]
    go_, po_, pl_, co_, own_, qo_ = (k[1] for k in keep)
    return lib.kvr_shared_query_attention(h, len(go) - 1 if n is None else n, go_, po_, pl_, pk, pv, co_, own_, qo_, q,
                                          kq, vq, ck, cv, out, ctypes.c_float(scale), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(go=(1, 2)), 1), (dict(go=(0, 2, 1), po=(0, 1, 2), pl=(0, 0)), 1), (dict(po=None), 1),
    (dict(po=(5, 2)), 1), (dict(pl=None), 1), (dict(pl=(101,)), 2), (dict(pl=(-1,)), 2), (dict(co=(0, 5, 4)), 1),
    (dict(own=None), 1), (dict(own=(20, 0)), 2), (dict(own=(-1, 0)), 2), (dict(qo=(0, 2, 1)), 1), (dict(qo=None), 1),
    (dict(q=None), 1), (dict(q=C + 2), 1), (dict(kq=None), 1), (dict(ck=Dp + 8), 1), (dict(out=None), 1),
    (dict(pk=None), 1), (dict(pv=Bp + 2), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(ck=A), 1), (dict(out=Bp), 1), (dict(cv=A + 128 * 2 * 4 * 99), 1),
    (dict(cv=Dp), 1), (dict(cv=Dp + 128 * 2 * 4 * 39), 1), (dict(out=E + 64), 1),
])
def test_shared_query_attention_refuses(lib, pool, kw, status):
    assert shared(lib, pool, **kw) == status
    assert lib.kvr_last_error().decode()


def test_shared_query_attention_with_nothing_to_do(lib, pool):
    assert shared(lib, None) == 1
    assert shared(lib, pool, n=0) == 0
    assert shared(lib, pool, go=(0, 0), co=(0,), own=(), qo=(0,)) == 0           # a group of no requests
    assert shared(lib, pool, qo=(0, 0, 0), q=None, pk=None) == 0                 # no query token
    if _no_gpu():
        assert shared(lib, pool) == 4
        assert shared(lib, pool, pl=(0,), pk=None, pv=None) == 4                 # nothing shared: no prefix needed


def test_shared_query_attention_positions_end_at_2_24(lib, pool):
    top = 1 << 24
    assert shared(lib, pool, po=(0, top), pl=(top - 4,), own=(3, 4)) == 2        # 4 own rows and one more


def weights(lib, h, co=(0, 20, 40), pl=(3, 4), qo=(0, 1, 2), q=A, ck=Bp, w=C, scale=0.0, flags=0, n=None):
    keep = [_p(co, np.int64), _p(pl, np.int32), _p(qo, np.int32)]
    return lib.kvr_key_weights(h, 2 if n is None else n, keep[0][1], keep[1][1], keep[2][1], q, ck, w,
                               ctypes.c_float(scale), flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(co=None), 1), (dict(co=(0, 9, 3)), 1), (dict(pl=None), 1), (dict(pl=(20, 0)), 2),
    (dict(pl=(-1, 0)), 2), (dict(qo=None), 1), (dict(qo=(0, 3, 1)), 1), (dict(q=None), 1), (dict(q=A + 8), 1),
    (dict(ck=None), 1), (dict(ck=Bp + 4), 1), (dict(w=None), 1), (dict(w=C + 2), 1), (dict(flags=2), 1),
    (dict(scale=-0.5), 1), (dict(w=Bp + 64), 1), (dict(w=A), 1),
])
def test_key_weights_refuses(lib, pool, kw, status):
    assert weights(lib, pool, **kw) == status
    assert lib.kvr_last_error().decode()


def test_key_weights_with_nothing_to_do(lib, pool):
    assert weights(lib, None) == 1
    assert weights(lib, pool, n=0) == 0
    assert weights(lib, pool, pl=(0, 0), qo=(0, 0, 0), q=None, ck=None, w=None) == 0
    assert weights(lib, pool, qo=(0, 0, 0), q=None, ck=None, w=None, flags=1) == 0   # nothing to add
    if _no_gpu():
        assert weights(lib, pool) == 4
        assert weights(lib, pool, qo=(0, 0, 0), q=None) == 4                         # zeros are written


def evict(lib, h, co=(0, 20, 40), n=(15, 20), keep=(8, 8), first=1, recent=2, w=A, ck=Bp, cv=C, do=(0, 10, 20), dk=Dp,
          dv=E, dw=F, kept=F + 0x1000000, flags=0, batch=None):
    k = [_p(co, np.int64), _p(n, np.int32), _p(keep, np.int32), _p(do, np.int64)]
    return lib.kvr_evict(h, 2 if batch is None else batch, k[0][1], k[1][1], k[2][1], first, recent, w, ck, cv, k[3][1],
                         dk, dv, dw, kept, flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(co=None), 1), (dict(do=None), 1), (dict(do=(0, 9, 8)), 1), (dict(n=None), 1),
    (dict(keep=None), 1), (dict(n=(21, 0)), 2), (dict(n=(-1, 0)), 2), (dict(keep=(2, 8)), 1), (dict(keep=(-1, 8), first=0, recent=0), 1),
    (dict(first=-1), 1), (dict(recent=-1), 1), (dict(first=1 << 30, recent=1 << 30), 1), (dict(keep=(11, 8)), 2), (dict(w=None), 1),
    (dict(w=A + 2), 1), (dict(ck=None), 1), (dict(cv=C + 8), 1), (dict(dk=None), 1), (dict(dv=E + 2), 1),
    (dict(dw=F + 1), 1), (dict(kept=None), 1), (dict(kept=F + 0x1000002), 1), (dict(flags=2), 1),
    (dict(dk=Bp), 1),                         # its own source, at other offsets
    (dict(dk=Bp + 256, do=(0, 20, 40)), 1),   # half over its source
    (dict(dk=C), 1), (dict(dv=Bp), 1), (dict(dw=A), 1), (dict(kept=A), 1), (dict(dk=E), 1), (dict(kept=Dp), 1),
])
def test_evict_refuses(lib, pool, kw, status):
    assert evict(lib, pool, **kw) == status
    assert lib.kvr_last_error().decode()


def test_evict_with_nothing_to_do(lib, pool):
    assert evict(lib, None) == 1
    assert evict(lib, pool, batch=0) == 0
    assert evict(lib, pool, co=(0, 0, 0), n=(0, 0), do=(0, 0, 0), w=None, ck=None, cv=None, dk=None, dv=None, dw=None,
                 kept=None) == 0
    if _no_gpu():
        assert evict(lib, pool) == 4
        assert evict(lib, pool, do=(0, 20, 40), dk=Bp, dv=C, dw=A) == 4      # in place
        assert evict(lib, pool, dw=None) == 4


def test_python_binding_checks_lengths_and_types():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    k = torch.zeros((1, 1, 1, 8, 64))
    p = kvr.Pool(k, k.clone(), 2, 1e4)
    x = torch.zeros(64)
    try:
        with pytest.raises(ValueError, match="own_len"):
            p.shared_query_attention([0, 1], [0, 4], [4], x, x, [0, 8], [], [0, 1], x, x, x, x, x, x, stream=0)
        with pytest.raises(ValueError, match="prefix_len"):
            p.key_weights([0, 8], [1, 2], [0, 1], x, x, x, stream=0)
        with pytest.raises(ValueError, match="float32"):
            p.key_weights([0, 8], [1], [0, 1], x, x, x.double(), stream=0)
        with pytest.raises(ValueError, match="keep"):
            p.evict([0, 8], [4], [2, 2], x, x, x, x.int(), stream=0)
        with pytest.raises(ValueError, match="int32"):
            p.evict([0, 8], [4], [2], x, x, x, x, stream=0)
        with pytest.raises(ValueError, match="dst_offsets"):
            p.evict([0, 8], [4], [2], x, x, x, x.int(), dst_k=x, stream=0)
        with pytest.raises(ValueError, match="dst_k"):
            p.evict([0, 8], [4], [2], x, x, x, x.int(), dst_v=x, stream=0)
    finally:
        p.close()


def _exchange_goes_wrong(ctas, blocks, bars):
    """Whether some order of steps lets a CTA read a pair that has not come.
    One thread a CTA; per row block it writes its pair to every CTA and arrives
    at that CTA's barrier, in turn, then waits for its own barrier's phase and
    reads all pairs.  Row block b uses barrier b % bars and its phase b // bars,
    of which a wait sees the parity alone, and the places b % 2."""
    state = (((0, 0),) * ctas, (((0, ctas),) * bars,) * ctas, (((-1,) * ctas,) * 2,) * ctas)
    seen, todo = {state}, [state]
    put = lambda t, i, x: t[:i] + (x,) + t[i + 1:]
    while todo:
        threads, barriers, places = todo.pop()
        for t, (b, x) in enumerate(threads):
            if b == blocks:
                continue
            k = b % bars
            if x < ctas:    # write to CTA x, arrive there
                done, left = barriers[x][k]
                done, left = (done + 1, ctas) if left == 1 else (done, left - 1)
                new = (put(threads, t, (b, x + 1)), put(barriers, x, put(barriers[x], k, (done, left))),
                       put(places, x, put(places[x], b % 2, put(places[x][b % 2], t, b))))
            else:
                if barriers[t][k][0] % 2 == (b // bars) % 2:
                    continue    # the phase is not complete
                if any(p != b for p in places[t][b % 2]):
                    return True
                new = (put(threads, t, (b + 1, 0)), barriers, places)
            if new not in seen:
                seen.add(new)
                todo.append(new)
    return False


def test_exchange_of_row_sums_between_ctas():
    """The window kernel's exchange: one barrier for all row blocks lets a CTA go
    on without a pair as soon as three CTAs take part; two by turns do not."""
    assert _exchange_goes_wrong(3, 2, 1)
    for ctas, blocks in ((2, 5), (3, 4), (4, 3)):
        assert not _exchange_goes_wrong(ctas, blocks, 2)


@pytest.mark.parametrize("kw", [dict(ck=C), dict(cv=C + 1024), dict(kq=Dp), dict(vq=E + 128 * 2 * 4 * 39),
                                dict(q=F - 4096, out=F - 4096 + 2048), dict(q=F, out=F - 256)])
def test_shared_query_attention_refuses_outputs_over_its_inputs(lib, pool, kw):
    """Other rows of the inputs are read while rows are written."""
    assert shared(lib, pool, **kw) == 1
    assert "overlap" in lib.kvr_last_error().decode()


def test_shared_query_attention_takes_its_queries_place(lib, pool):
    """The output in the queries' own buffer: each row is read before it is written."""
    if _no_gpu():
        assert shared(lib, pool, q=F, out=F) == 4


def test_python_binding_refuses_lengths_that_are_not_integers():
    """Nothing is cut to an integer or to 32 bits on the way."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    assert [list(kvr._ints("x", a, "i")[0]) for a in ([1, 2], (1, 2), np.array([1, 2], np.int64), torch.tensor([1, 2]))] == [[1, 2]] * 4
    assert list(kvr._ints("x", np.array([1 << 40]), "q")[0]) == [1 << 40]
    assert kvr._ints("x", np.array([]), "i")[2] == 0
    for a in (np.array([1.5, 2.0]), np.array([1.0]), np.array([(1 << 32) + 5]), np.array([1 << 31], np.uint32), torch.tensor([0.5]),
              np.array([True])):
        with pytest.raises(ValueError, match="x must hold 32-bit integers"):
            kvr._ints("x", a, "i")
    for a in ([1.5], [1 << 31]):
        with pytest.raises((TypeError, OverflowError)):
            kvr._ints("x", a, "i")
    k = torch.zeros((1, 1, 1, 8, 64))
    p, x = kvr.Pool(k, k.clone(), 2, 1e4), torch.zeros(64)
    try:
        with pytest.raises(ValueError, match="group_offsets"):
            p.shared_query_attention([], [0], [], x, x, [0], [], [0], x, x, x, x, x, x, stream=0)
        with pytest.raises(kvr.KvrError) as e:
            p.shared_query_attention([0, -1], [0, 4], [4], x, x, [0], [], [0], x, x, x, x, x, x, stream=0)
        assert e.value.status == 1
    finally:
        p.close()


def test_python_binding_refuses_tensors_that_a_call_would_leave():
    """Another type, a strided view, too few values, pageable memory: refused by
    name, for every tensor of the three calls."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D = 2, 2, 3, 64
    k = torch.zeros((1, L, H, 8, D))
    p = kvr.Pool(k, k.clone(), H * G, 1e4)
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt)
    row = L * H * D
    shared = dict(prefix_k=z(30 * row), prefix_v=z(30 * row), q=z(3 * L * H * G * D), kq=z(3 * L * H * D), vq=z(3 * L * H * D),
                  cache_k=z(20 * row), cache_v=z(20 * row), out=z(3 * L * H * G * D))
    weights = dict(q=z(3 * L * H * G * D), cache_k=z(20 * row), weights=z(20 * L * H))
    evict = dict(weights=z(20 * L * H), cache_k=z(20 * row), cache_v=z(20 * row), kept=z(9 * L * H, torch.int32), dst_k=z(12 * row),
                 dst_v=z(12 * row), dst_weights=z(12 * L * H))
    calls = ((shared, lambda **t: p.shared_query_attention([0, 2], [0, 30], [25], cache_offsets=[0, 10, 20], own_len=[2, 3],
                                                           q_offsets=[0, 1, 3], stream=0, **t)),
             (weights, lambda **t: p.key_weights([0, 10, 20], [2, 3], [0, 1, 3], stream=0, **t)),
             (evict, lambda **t: p.evict([0, 10, 20], [8, 7], [5, 4], dst_offsets=[0, 6, 12], stream=0, **t)))
    try:
        for good, call in calls:
            for name, t in good.items():
                for bad, why in ((t.double(), "contiguous"), (torch.zeros(2 * t.numel(), dtype=t.dtype)[::2], "contiguous"),
                                 (t[:-1].clone(), "at least")):
                    pinned = {n: _Pinned(x) for n, x in good.items()}   # (no device here)
                    with pytest.raises(ValueError, match=f"{name} must .*{why}"):
                        call(**dict(pinned, **{name: _Pinned(bad)}))
                if not t.is_pinned():
                    with pytest.raises(ValueError, match=f"{name} must be in device or pinned"):
                        call(**dict({n: _Pinned(x) for n, x in good.items()}, **{name: t}))
        if _no_gpu():   # the tensors as they should be reach the library
            for good, call in calls:
                with pytest.raises(kvr.KvrError) as e:
                    call(**{n: _Pinned(x) for n, x in good.items()})
                assert e.value.status == 4
    finally:
        p.close()


class _Pinned:
    """A tensor that says it is in pinned memory."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return (lambda: True) if name == "is_pinned" else getattr(self.t, name)


def test_shared_tables_are_the_same_from_lists_and_arrays():
    from rag_precomputed_kv_gb300 import kvr
    read = lambda a, m, kind: np.ctypeslib.as_array((kind * m).from_address(a)).tolist() if m else []
    for tables in (([0, 2, 2, 5], [3, 10, 14, 1 << 40], [7, 0, 9], [0, 4, 9, 12, 15, 1 << 35], [1, 2, 3, 0, 5], [0, 1, 1, 4, 5, 9]),
                   ([0, 0], [0, 4], [4], [0], [], [0]), ([0], [0], [], [0], [], [0])):
        want = [list(x) for x in tables]
        for args in (tables, [np.array(x, np.int64) for x in tables], [tuple(x) for x in tables]):
            keep, n, tokens, rows, pre, *addr = kvr._shared_tables(*args)
            b = tables[0][-1]
            assert (n, tokens, rows) == (len(tables[0]) - 1, tables[5][-1], tables[3][-1])
            assert pre == (tables[1][-1] if any(tables[2]) else 0)
            assert [read(a, m, k) for a, m, k in zip(addr, (n + 1, n + 1, n, b + 1, b, b + 1),
                                                     (ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                                      ctypes.c_int32))] == want
    with pytest.raises(ValueError, match="own_len must hold 2"):
        kvr._shared_tables([0, 2], [0, 4], [4], [0, 1, 2], [1], [0, 1, 2])
    with pytest.raises((TypeError, OverflowError)):
        kvr._shared_tables([0, 1], [0, 4], [4.5], [0, 1], [1], [0, 1])


def test_shared_path_before_any_call(lib, pool):
    from rag_precomputed_kv_gb300 import kvr
    assert lib.kvr_shared_path(None) == -2
    assert lib.kvr_shared_path(pool) == kvr.SHARED_NONE
