"""The paged cache on the CPU: every refused argument is refused with a status,
before any GPU work; the binding's own checks; the packed format's rounding."""
import ctypes
import glob
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from rag_precomputed_kv_gb300 import build as B

A, Bp, C, Dp, E, F = (0x10000000 * (i + 1) for i in range(6))   # far apart, aligned
L, H, G, D = 2, 2, 4, 128
ROW, UNIT = D, 64 * D
TOP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    B.build()
    from rag_precomputed_kv_gb300 import kvr
    return kvr.load()


def _register(lib, dtype, d):
    from rag_precomputed_kv_gb300 import kvr
    desc = kvr.PoolDesc(L, H * G, H, d, dtype, 0, 4, 512, 0x10000, 0x20000, (ctypes.c_int64 * 4)(L * H * 512 * d, H * 512 * d, 512 * d, d), 1e6)
    h = ctypes.c_void_p()
    assert lib.kvr_pool_register(ctypes.byref(desc), ctypes.byref(h)) == 0
    return h


@pytest.fixture(scope="module")
def pool(lib):
    h = _register(lib, 0, 128)
    yield h
    lib.kvr_pool_unregister(h)


@pytest.fixture(scope="module")
def pool32(lib):
    h = _register(lib, 1, 64)
    yield h
    lib.kvr_pool_unregister(h)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


def _p(x, dt=np.int32):
    if x is None:
        return None, None
    a = np.ascontiguousarray(x, dt)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _pages(k=A, v=Bp, n=8, rows=64, stride=(L * H * UNIT, H * UNIT, UNIT)):
    from rag_precomputed_kv_gb300 import kvr
    return kvr.PageDesc(k, v, n, rows, (ctypes.c_int64 * 3)(*stride))


def _packed(data=C, n=8):
    from rag_precomputed_kv_gb300 import kvr
    return kvr.PackedDesc(data, n)


def _ref(x):
    return None if x is None else ctypes.byref(x)


BAD_PAGES = [
    (dict(pages=None), 1), (dict(pages=dict(k=None)), 1), (dict(pages=dict(v=Bp + 8)), 1), (dict(pages=dict(n=0)), 1),
    (dict(pages=dict(n=1 << 31)), 1), (dict(pages=dict(rows=0)), 1), (dict(pages=dict(rows=TOP + 1)), 1),
    (dict(pages=dict(stride=(-64, H * UNIT, UNIT))), 1), (dict(pages=dict(stride=(L * H * UNIT + 4, H * UNIT, UNIT))), 1),
    (dict(pages=dict(stride=(1 << 60, H * UNIT, UNIT))), 1),
]
ON_EACH_OTHER = [
    (dict(pages=dict(stride=(0, H * UNIT, UNIT))), 1), (dict(pages=dict(stride=(L * H * UNIT, H * UNIT, UNIT - 128))), 1),
    (dict(pages=dict(stride=(L * H * UNIT, UNIT, UNIT))), 1),
]
BAD_TABLE = [
    (dict(n=-1), 1), (dict(width=-1), 1), (dict(table=None), 1), (dict(table=((8, 1), (2, 3))), 2), (dict(table=((-1, 1), (2, 3))), 2),
]


def append(lib, h, pages={}, table=((0, 1), (2, 3)), width=2, start=(10, 60), qo=(0, 1, 9), k=C, v=Dp, stride=None, flags=0, n=None):
    pg = None if pages is None else _pages(**pages)
    t, s, q, st = _p(table), _p(start), _p(qo), _p(stride, np.int64)
    return lib.kvr_page_append(h, _ref(pg), 2 if n is None else n, t[1], width, s[1], q[1], k, v, st[1], flags, None)


@pytest.mark.parametrize("kw,status", BAD_PAGES + ON_EACH_OTHER + BAD_TABLE + [
    (dict(start=None), 1), (dict(qo=None), 1), (dict(qo=(0, 2, 1)), 1), (dict(qo=(1, 2, 3)), 1), (dict(k=None), 1), (dict(v=Dp + 2), 1),
    (dict(flags=2), 1), (dict(start=(-1, 0)), 2), (dict(start=(10, 121)), 2), (dict(start=(TOP, 0)), 2),
    (dict(table=((0, 1), (0, 3))), 1),                       # one page, two requests
    (dict(table=((0, 1), (2, 2))), 1),                       # twice in one
    (dict(stride=(1024, 4, 128)), 1), (dict(stride=(-8, 256, 128)), 1), (dict(stride=(1 << 60, 256, 128)), 1),
    (dict(k=A + 2 * UNIT), 1), (dict(v=Bp), 1),              # new rows among the pages
])
def test_append_refuses(lib, pool, kw, status):
    assert append(lib, pool, **kw) == status
    assert lib.kvr_last_error().decode()


def test_append_with_nothing_to_do_and_pages_it_does_not_read(lib, pool):
    assert append(lib, None) == 1
    assert append(lib, pool, n=0, qo=(0,), start=None, table=None) == 0
    assert append(lib, pool, qo=(0, 0, 0), k=None, v=None, table=None) == 0
    if _no_gpu():
        assert append(lib, pool) == 4
        # pages without new rows are not looked at: one that another request writes, none at all
        assert append(lib, pool, table=((0, -5), (2, 3))) == 4
        assert append(lib, pool, start=(10, 64), table=((0, 3), (0, 3))) == 4
        assert append(lib, pool, pages=dict(n=1, stride=(0, H * UNIT, UNIT)), table=((0, 0), (0, 0)), qo=(0, 1, 1)) == 4   # one page
        # a flat block [L][H][256][D] as four pages
        assert append(lib, pool, pages=dict(n=4, stride=(UNIT, H * 4 * UNIT, 4 * UNIT))) == 4


def attend(lib, h, pages={}, table=((0, 1), (2, 3)), width=2, kv=(100, 128), pos=None, qo=(0, 1, 9), q=C, out=Dp, window=0, first=0,
           packed=None, ptable=((0, 1), (2, 3)), pwidth=2, plen=(64, 96), scale=0.0, n=None):
    pg = None if pages is None else _pages(**pages)
    pk = None if packed is None else _packed(**packed)
    t, kl, qp, qof = _p(table), _p(kv), _p(pos), _p(qo)
    pt, pl = (_p(ptable), _p(plen)) if pk is not None else (_p(None), _p(None))
    return lib.kvr_page_attention(h, _ref(pg), 2 if n is None else n, t[1], width, kl[1], qp[1], qof[1], q, out, window, first,
                                  _ref(pk), pt[1], pwidth, pl[1], ctypes.c_float(scale), None)


PACK = dict(data=E)


@pytest.mark.parametrize("kw,status", BAD_PAGES + BAD_TABLE + [
    (dict(kv=None), 1), (dict(kv=(-1, 5)), 2), (dict(kv=(129, 128)), 2), (dict(kv=(0, 128)), 2),   # (a token before row 0)
    (dict(pos=(-1, 0)), 2), (dict(pos=(TOP, 0)), 2), (dict(qo=None), 1), (dict(qo=(0, 2, 1)), 1), (dict(q=None), 1),
    (dict(q=C + 8), 1), (dict(out=None), 1), (dict(out=Dp + 2), 1), (dict(window=-1), 1), (dict(first=-1), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(out=A + 64), 1), (dict(out=Bp), 1), (dict(out=C + 256), 1),
    (dict(packed=dict(data=None)), 1), (dict(packed=dict(data=E + 8)), 1), (dict(packed=dict(data=E, n=0)), 1),
    (dict(packed=PACK, plen=None), 1), (dict(packed=PACK, ptable=None), 1), (dict(packed=PACK, plen=(65, 0)), 2),
    (dict(packed=PACK, plen=(-32, 0)), 2), (dict(packed=PACK, plen=(128, 0)), 2), (dict(packed=PACK, ptable=((0, 8), (2, 8))), 2),
    (dict(packed=PACK, pwidth=0), 2), (dict(packed=PACK, pages=dict(rows=48)), 1), (dict(packed=dict(data=Dp)), 1),
])
def test_attention_refuses(lib, pool, kw, status):
    assert attend(lib, pool, **kw) == status
    assert lib.kvr_last_error().decode()


def test_attention_with_nothing_to_do_and_pages_it_does_not_read(lib, pool, pool32):
    assert attend(lib, None) == 1
    assert attend(lib, pool, n=0, qo=(0,), kv=None, table=None) == 0
    assert attend(lib, pool, qo=(0, 0, 0), q=None, out=None, table=None) == 0
    assert attend(lib, pool32, packed=PACK, pages=dict(stride=(L * H * 64 * 64, H * 64 * 64, 64 * 64))) == 3   # fp32: not packed
    if _no_gpu():
        assert attend(lib, pool) == 4
        assert attend(lib, pool, out=C) == 4                                                   # in place
        assert attend(lib, pool, table=((0, 0), (0, 0))) == 4                                  # shared pages
        assert attend(lib, pool, kv=(0, 0), pos=(0, 7), table=None) == 4                       # nothing to see
        assert attend(lib, pool, window=36, table=((-1, 1), (7, 7))) == 4                      # rows 64 .. 99; 84 .. 127
        assert attend(lib, pool, window=37, table=((-1, 1), (7, 7))) == 2
        assert attend(lib, pool, window=30, first=1, table=((-1, 1), (7, 7))) == 2
        assert attend(lib, pool, packed=PACK, table=((-1, 1), (-1, 3))) == 4                   # rows 0 .. 63 are packed
        assert attend(lib, pool, packed=PACK, plen=(32, 96), table=((-1, 1), (-1, 3))) == 2
        assert attend(lib, pool, pages=dict(stride=(0, 0, 0))) == 4                            # read only: rows may be shared


def pack(lib, h, pages={}, table=((0, 1), (2, 3)), width=2, packed={}, ptable=((0, 1), (2, 3)), pwidth=2, begin=(0, 32), end=(64, 96),
         n=None, unpack=False):
    pg = None if pages is None else _pages(**pages)
    pk = None if packed is None else _packed(**packed)
    t, pt, b, e = _p(table), _p(ptable), _p(begin), _p(end)
    n = 2 if n is None else n
    if unpack:
        return lib.kvr_page_unpack(h, _ref(pk), n, pt[1], pwidth, _ref(pg), t[1], width, b[1], e[1], None)
    return lib.kvr_page_pack(h, _ref(pg), n, t[1], width, _ref(pk), pt[1], pwidth, b[1], e[1], None)


@pytest.mark.parametrize("unpack", [False, True])
@pytest.mark.parametrize("kw,status", BAD_PAGES + BAD_TABLE + [
    (dict(packed=None), 1), (dict(packed=dict(data=None)), 1), (dict(packed=dict(data=C + 8)), 1), (dict(packed=dict(n=0)), 1),
    (dict(pages=dict(rows=40)), 1), (dict(pwidth=-1), 1), (dict(ptable=None), 1), (dict(ptable=((9, 1), (2, 3))), 2),
    (dict(packed=dict(n=(1 << 31) - 1), pages=dict(rows=TOP, stride=(1 << 27, 1 << 27, 1 << 27), n=1)), 1),   # more bytes than there are
    (dict(begin=None), 1), (dict(end=None), 1), (dict(begin=(1, 32)), 1), (dict(end=(33, 96)), 1), (dict(end=(64, 0)), 1),
    (dict(begin=(-32, 0)), 1), (dict(end=(160, 96)), 2), (dict(end=(TOP + 32, 96)), 1), (dict(packed=dict(data=A)), 1),
    (dict(packed=dict(data=Bp + 4608)), 1),
])
def test_pack_refuses(lib, pool, kw, status, unpack):
    assert pack(lib, pool, unpack=unpack, **kw) == status
    assert lib.kvr_last_error().decode()


def test_pack_writes_each_page_once(lib, pool, pool32):
    twice = ((0, 1), (0, 3))
    assert pack(lib, pool, ptable=twice) == 1 and pack(lib, pool, table=twice, unpack=True) == 1
    for kw, status in ON_EACH_OTHER:
        assert pack(lib, pool, unpack=True, **kw) == status
    assert pack(lib, None) == 1 and pack(lib, pool, n=0) == 0 and pack(lib, pool, begin=(0, 32), end=(0, 32), table=None, ptable=None) == 0
    assert pack(lib, pool32, pages=dict(stride=(L * H * 64 * 64, H * 64 * 64, 64 * 64))) == 3
    if _no_gpu():
        assert pack(lib, pool) == 4 and pack(lib, pool, unpack=True) == 4
        assert pack(lib, pool, table=twice) == 4 and pack(lib, pool, ptable=twice, unpack=True) == 4   # read twice


def test_packed_page_bytes(lib, pool, pool32):
    assert lib.kvr_packed_page_bytes(pool, 64) == L * H * 2 * 4608
    assert [lib.kvr_packed_page_bytes(pool, r) for r in (0, -32, 33, TOP + 32)] == [0] * 4
    assert lib.kvr_packed_page_bytes(pool32, 64) == 0 and lib.kvr_packed_page_bytes(None, 64) == 0


def test_no_code_depends_on_how_the_quotient_is_rounded():
    """x and the scale have 8 significant bits: a quotient that is not exactly
    between two codes is at least 2^-10 away from the middle, whatever the exponents."""
    gap = Fraction(1)
    for b in range(128, 256):
        for a in range(128, 256):
            for d in range(-4, 4):
                x = Fraction(a, b) * Fraction(2) ** d
                if x <= 8:
                    away = abs(x - (x - Fraction(1, 2)).__round__() - Fraction(1, 2))
                    if away:
                        gap = min(gap, away)
    assert gap >= Fraction(1, 1024)


def test_binding_checks():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    t = torch.zeros((2, 3), dtype=torch.int32)
    assert kvr._page_table("t", t, 2)[1:] == (t.data_ptr(), 3)                     # as it is
    assert kvr._page_table("t", [[1, 2], [3]], 2)[0].tolist() == [[1, 2], [3, -1]]
    assert kvr._page_table("t", t[:, :2], 2)[0].tolist() == [[0, 0], [0, 0]]
    assert kvr._page_table("t", None, 2) == (None, None, 0)
    assert kvr._page_table("t", [], 0)[2] == 0
    for bad, n in ((t, 3), (t[0], 2), (np.zeros((2, 2)) + 0.5, 2), (np.full((1, 1), 1 << 40), 1)):
        with pytest.raises(ValueError):
            kvr._page_table("t", bad, n)
    k = torch.zeros((2, 1, 2, 16, 64))
    for a, b in ((k, k[:1]), (k, k.bfloat16()), (k[0], k[0]), (k.transpose(3, 4), k.transpose(3, 4)), (k[..., :32], k[..., :32]), (k, k)):
        with pytest.raises(ValueError):   # (the last: host memory)
            kvr.Pages(a, b)
    for d in (torch.zeros(4, dtype=torch.uint8), torch.zeros((2, 4)), torch.zeros((2, 4), dtype=torch.uint8)):
        with pytest.raises(ValueError):
            kvr.PackedPages(d, 32)


def test_keys_that_are_the_values_are_read_but_not_written(lib, pool):
    same = dict(pages=dict(v=A))
    assert append(lib, pool, **same) == 1
    assert "same rows" in lib.kvr_last_error().decode()
    assert pack(lib, pool, unpack=True, **same) == 1
    if _no_gpu():
        assert attend(lib, pool, **same) == 4
        assert pack(lib, pool, **same) == 4


def test_keys_and_values_that_lie_upon_each_other_are_read_but_not_written(lib, pool):
    """v some elements, rows, pages, heads or layers behind k (or before it) in one dense pool; and side by
    side in one tensor, which is fine."""
    page, layer = L * H * UNIT, H * UNIT
    for d in (8, 64, ROW, UNIT - ROW, UNIT, UNIT + 64, 2 * UNIT, layer, layer + UNIT, page - ROW, page, 7 * page, 8 * page - 64):
        for a, b in ((A, A + 2 * d), (A + 2 * d, A)):
            kw = dict(pages=dict(k=a, v=b))
            assert append(lib, pool, k=E, v=F, **kw) == 1 and "lie upon" in lib.kvr_last_error().decode(), d
            assert pack(lib, pool, unpack=True, **kw) == 1, d
            if _no_gpu():
                assert attend(lib, pool, q=E, out=F, **kw) == 4 and pack(lib, pool, **kw) == 4
    beside = [((2 * page, layer, UNIT), page), ((2 * page, 2 * layer, UNIT), layer), ((2 * page, 2 * layer, 2 * UNIT), UNIT),
              ((page, layer, UNIT), 8 * page), ((2 * UNIT, 16 * layer, 16 * UNIT), UNIT)]
    if _no_gpu():
        for stride, d in beside:
            for a, b in ((A, A + 2 * d), (A + 2 * d, A)):
                assert append(lib, pool, k=E, v=F, pages=dict(k=a, v=b, stride=stride)) == 4, (stride, d)
    for stride, d in beside[:3]:      # a row further on they meet
        assert append(lib, pool, k=E, v=F, pages=dict(k=A, v=A + 2 * (d + ROW), stride=stride)) == 1


@pytest.mark.skipif("not _no_gpu()")
def test_where_rows_lie_is_found_as_by_trying_all(lib, pool):
    rng = np.random.default_rng(1)
    seen = [0, 0]
    for _ in range(400):
        n, rows = int(rng.integers(1, 5)), int(rng.integers(1, 3))
        run, stride = rows * ROW, [0, 0, 0]
        need = run
        for i in rng.permutation(3):
            stride[i] = need * int(rng.integers(1, 5)) + 8 * int(rng.integers(0, 20))
            need += ((n, L, H)[i] - 1) * stride[i]
        d = 8 * int(rng.integers(-need // 8 - 2, need // 8 + 3))
        starts = (np.arange(n)[:, None, None] * stride[0] + np.arange(L)[:, None] * stride[1] + np.arange(H) * stride[2]).ravel()
        meet = bool((np.abs(starts[:, None] - starts[None] - d) < run).any())
        seen[meet] += 1
        got = append(lib, pool, pages=dict(k=A + (1 << 20), v=A + (1 << 20) + 2 * d, n=n, rows=rows, stride=tuple(stride)), table=((0,), (0,)),
                     width=1, start=(0, 0), qo=(0, 1, 1), k=E, v=F)
        assert got == (1 if meet else 4), (n, rows, stride, d)
    assert min(seen) > 50


def test_binding_refuses_numbers_that_it_would_have_to_cut(lib, pool):
    import torch
    from rag_precomputed_kv_gb300 import kvr
    own, pages = object.__new__(kvr.Pool), object.__new__(kvr.Pages)
    own.__dict__.update(_h=pool, n_layers=L, n_kv_heads=H, n_q_heads=H * G, head_dim=D, dtype=torch.bfloat16, _layout=(L, H, D), _wide=H * G * D)
    desc = _pages()
    pages.__dict__.update(shape=(L, H, D), dtype=torch.bfloat16, page_rows=64, _d=desc, _p=ctypes.addressof(desc))
    try:
        def call(**kw):
            own.page_attention(pages, [[0]], [0], [0, 0], None, None, stream=0, **kw)

        for name in ("window", "n_first"):
            for x in (0, 5, np.int64(7), (1 << 31) - 1):
                call(**{name: x})
            for x in (2.5, 1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 33), "3"):
                with pytest.raises((TypeError, ValueError)):
                    call(**{name: x})
            with pytest.raises(kvr.KvrError):
                call(**{name: -1})
        assert own.packed_page_bytes(64) == lib.kvr_packed_page_bytes(pool, 64)
        for x in ((1 << 32) + 64, 64.5):
            with pytest.raises((TypeError, ValueError)):
                own.packed_page_bytes(x)
    finally:
        own._h = None
    for bad in ([[1.5, 2]], [[1, 2.0]], [[1 << 40]], [[1], [None]]):
        with pytest.raises((TypeError, ValueError, OverflowError)):
            kvr._page_table("t", bad, len(bad))
    assert kvr._page_table("t", [(np.int32(4), 2), []], 2)[0].tolist() == [[4, 2], [-1, -1]]
    assert kvr._page_table("t", [[], []], 2)[2] == 0


def test_what_host_threads_share_is_atomic():
    """Two pools may be called by two threads at once: what a launcher keeps between calls is constant or atomic."""
    kept = re.compile(r"^\s+static (?!const\b|constexpr\b|std::atomic<)[^(;={]*(?:;|=|\{)", re.M)
    found = {}
    for path in glob.glob(os.path.join(B.CSRC, "*.cu*")):
        with open(path) as f:
            found[os.path.basename(path)] = kept.findall(re.sub(r"//[^\n]*", "", f.read()))
    assert len(found) > 10 and not {k: v for k, v in found.items() if v}
    assert kept.findall("    static int caps[64];\n    static bool x = 1;\n    static std::atomic<int> y;\n    static kvr_status f(int a);\n") == [
        "    static int caps[64];", "    static bool x ="]


def test_limits_of_the_accuracy_tests_tell_the_roundings_apart():
    """The model behind the limits of the GPU tests' norms, in fp64 with operands rounded to bf16 here: an error
    in units of the output's own rounding, squared, is the number of roundings, and one more passes no limit."""
    import torch
    bf = lambda x: x.to(torch.bfloat16).double()

    def roundings(packed):
        g = torch.Generator().manual_seed(3)
        off = dict.fromkeys(("none", "q", "p", "qp", "qpkv"), 0.0)
        own = 0.0
        for _ in range(8):
            q = torch.randn((32, 128), generator=g).double()
            k, v = (bf(torch.randn((700, 128), generator=g)) for _ in range(2))
            if packed:
                k, v = ((torch.round(y / s).clamp(-7, 7) * s).view(700, 128)
                        for y, s in ((x.view(700, 4, 32), bf(x.view(700, 4, 32).abs().amax(-1, keepdim=True) / 7)) for x in (k, v)))

            def out(r=""):
                a, b, c = (bf(x) if y in r else x for x, y in ((q, "q"), (k, "k"), (v, "v")))
                s = a @ b.T * 128 ** -0.5
                p = torch.exp(s - s.amax(-1, keepdim=True))
                return (bf(p) if "p" in r else p) @ c / p.sum(-1, keepdim=True)

            want = out()
            own += float((bf(want) - want).norm() ** 2)
            for r in off:
                off[r] += float((bf(out(r.replace("none", ""))) - want).norm() ** 2)
        return {r: x / own for r, x in off.items()}

    n = roundings(False)      # limits: 1 + 1/2, 3 + 1/2
    assert n["none"] < 1.01 and 1.5 < n["q"] < 2.5 and 1.5 < n["p"] < 2.5 and 2.5 < n["qp"] < 3.5, n
    n = roundings(True)       # 2 + 1/2, 5 + 1/2
    assert 1.5 < n["p"] < 2.5 < n["qp"] < 3.5 < n["qpkv"] < 5.5, n


def test_page_path_before_any_call(lib, pool):
    from rag_precomputed_kv_gb300 import kvr
    assert lib.kvr_page_path(None) == -2
    assert lib.kvr_page_path(pool) == kvr.PAGE_NONE


def test_binding_refuses_queries_padded_on_the_token_axis(lib, pool):
    """[layers, more tokens than the offsets say, heads, head_dim]: its layers are not where the library takes them."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    own, pages = object.__new__(kvr.Pool), object.__new__(kvr.Pages)
    own.__dict__.update(_h=pool, n_layers=L, n_kv_heads=H, n_q_heads=H * G, head_dim=D, dtype=torch.bfloat16, _layout=(L, H, D), _wide=H * G * D)
    desc = _pages()
    pages.__dict__.update(shape=(L, H, D), dtype=torch.bfloat16, page_rows=64, _d=desc, _p=ctypes.addressof(desc))
    right, wide = (torch.zeros((L, n, H * G, D), dtype=torch.bfloat16) for n in (3, 5))
    try:
        for q, out in ((wide, right), (right, wide), (wide, wide)):
            with pytest.raises(ValueError, match="must hold 3 tokens in each layer"):
                own.page_attention(pages, [[0]], [9], [0, 3], q, out, stream=0)
        for q in (right, wide.view(-1), wide.view(L, -1)):      # (as it should be, and buffers without a token axis: on to the next check)
            with pytest.raises(ValueError, match="device memory"):
                own.page_attention(pages, [[0]], [9], [0, 3], q, right, stream=0)
        own.n_layers = 1                                        # one layer: tokens behind the last are left alone
        with pytest.raises(ValueError, match="device memory"):
            own.page_attention(pages, [[0]], [9], [0, 3], wide[:1], right[:1], stream=0)
    finally:
        own._h = None
