"""Paged cache: what a call uses beside its arguments."""
import threading

import numpy as np
import pytest

from test_gpu_page_accuracy import _attend64, _off, _turn64
from test_gpu_page_cache import _pool, _randn, _starts, _table

pytestmark = pytest.mark.gpu


def test_two_threads_with_a_pool_each():
    """Calls of every kernel from two host threads at once, each on its own pool, stream and pages."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R, n = 2, 2, 4, 128, 32, 400
    t, pages = _table([n], R, 3)
    jobs = []
    for i in range(2):
        k, v = _randn(10 * i, (pages, L, H, R, D), "bf16"), _randn(10 * i + 1, (pages, L, H, R, D), "bf16")
        jobs.append([kvr.Pages(k, v), _randn(10 * i + 2, (L, 60, H * G, D), "bf16"), _randn(10 * i + 3, (L, 60, H, D), "bf16")])

    def work(job, pool, stream):
        out = []
        packed = pool.packed_pages(pages, R)
        pool.page_append(job[0], t, [n - 60], [0, 60], job[2], job[2], stream=stream)
        pool.page_pack(job[0], t, packed, t, [0], [320], stream=stream)
        for q in (1, 4, 12, 60):
            Q = job[1][:, :q].contiguous()
            for kw in ({}, dict(packed=packed, packed_table=t, packed_len=[320])):
                o = torch.empty_like(Q)
                pool.page_attention(job[0], t, [n], [0, q], Q, o, stream=stream, **kw)
                out.append(o)
        stream.synchronize()
        pool.check(stream=stream)
        return out

    want = [work(job, _pool(L, H, G, D, "bf16"), torch.cuda.current_stream()) for job in jobs]
    got, meet = [[], []], threading.Barrier(2)

    def thread(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                pool = _pool(L, H, G, D, "bf16")
                stream.synchronize()
                meet.wait(60)
                got[i].append(work(jobs[i], pool, stream))

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join(120)
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 5
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_restored_rows_in_slices_of_units():
    """64 query rows on packed rows, whose restored form passes the scratch's 1 GiB: two slices of
    the (layer, kv-head) units, the second a unit shorter, against fp64 unit by unit."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, D, R, n, q = 13, 5, 128, 128, 33152, 64
    pool = _pool(L, H, 1, D, "bf16")
    k, v = (_randn(i, (n // R, L, H, R, D), "bf16") for i in (1, 2))
    t = np.random.default_rng(0).permutation(n // R).astype(np.int32)[None]
    packed = pool.packed_pages(n // R, R)
    pages = kvr.Pages(k, v)
    pool.page_pack(pages, t, packed, t, [0], [n])
    Q = _randn(3, (L, q, H, D), "bf16")
    out = torch.full_like(Q, float("nan"))
    for _ in range(2):      # the second call meets the first one's scratch
        pool.page_attention(pages, t, [n], [0, q], Q, out, packed=packed, packed_table=t, packed_len=[n])
        pool.check()
    path = pool.page_path
    assert path & kvr.PAGE_RESTORED and path & kvr.PAGE_MANY and path >> 8 == 2
    # what the restoring kernel gives for each row, rounded to bf16: three roundings are left
    pool.page_unpack(packed, t, pages, t, [0], [n])
    pos = n - q + np.arange(q)
    turned = _turn64(Q.double(), pos)
    for l in range(L):
        K, V = (torch.cat([x[int(i), l] for i in t[0]], 1)[None].double() for x in (k, v))
        want = _attend64(turned[l:l + 1], K, V, pos, D ** -0.5)
        for h in range(H):
            off, r = _off(out[l, :, h], want[0, :, h])
            assert off <= r * np.sqrt(3 + 1), (l, h, off, r)


def test_which_kernels_ran():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    R = 32

    def path(reqs, G=4, D=128, dtype="bf16"):
        pool = _pool(1, 2, G, D, dtype)
        assert pool.page_path == kvr.PAGE_NONE
        kv, lq, body = (list(x) for x in zip(*reqs))
        t, n = _table(kv, R, 3)
        pages = kvr.Pages(*(_randn(i, (n, 1, 2, R, D), dtype) for i in (1, 2)))
        kw = {}
        if any(body):
            packed = pool.packed_pages(n, R)
            pool.page_pack(pages, t, packed, t, [0] * len(kv), body)
            kw = dict(packed=packed, packed_table=t, packed_len=body)
        Q = _randn(3, (1, sum(lq), 2 * G, D), dtype)
        pool.page_attention(pages, t, kv, _starts(lq).astype(np.int32), Q, Q, **kw)
        pool.check()
        return pool.page_path & 255, pool.page_path >> 8

    few, many, rest = kvr.PAGE_FEW, kvr.PAGE_MANY, kvr.PAGE_RESTORED
    assert path([(90, 4, 0)], D=64) == path([(90, 4, 0)], dtype="fp32") == (kvr.PAGE_CUDA_CORES, 0)
    assert path([(90, 4, 0)]) == path([(90, 4, 64), (90, 1, 0)]) == path([(90, 12, 64)]) == (few, 0)
    assert path([(90, 5, 0)]) == (many, 1) and path([(90, 5, 0), (90, 12, 64)]) == (few | many, 1)
    assert path([(90, 13, 64)]) == (many | rest, 1) and path([(90, 13, 64), (90, 1, 0)]) == (few | many | rest, 1)
    assert path([(90, 1, 64)], G=20) == (many | rest, 1) and path([(90, 1, 0)], G=20) == (many, 1)
    assert path([(4000, 20, 0)], G=1) == (many | kvr.PAGE_JOINED, 1)


@pytest.mark.parametrize("G,reqs,fits", [
    (4, [(90, 4, 0)], True), (4, [(90, 5, 0)], False),                  # 16 query rows, and 20
    (4, [(90, 12, 64)], True), (4, [(90, 13, 64)], False),              # three parts, and four
    (7, [(90, 6, 64)], True), (7, [(90, 7, 64)], False),                # of two tokens each
    (16, [(90, 3, 32)], True), (20, [(90, 1, 0)], False), (20, [(90, 1, 32)], False),
    (4, [(40, 1, 0)] * 64, True), (4, [(40, 1, 0)] * 65, False),
    (4, [(40, 8, 32)] * 32, True), (4, [(40, 8, 32)] * 33, False),      # two parts each
    (4, [(512 * 32, 1, 512 * 32)] * 2, True), (4, [(512 * 32 + 1, 1, 512 * 32)] * 2, False),   # 1,024 page numbers; 2 more
    (4, [(1024 * 32, 1, 0)], True), (4, [(1025 * 32, 1, 0)], False),
])
def test_which_calls_can_be_captured(G, reqs, fits):
    import gc

    import torch
    from rag_precomputed_kv_gb300 import kvr
    H, D, R = 1, 128, 32
    pool = _pool(1, H, G, D, "bf16")
    pool.reserve(max_batch=128, max_spans=4096, max_query_tokens=256)
    kv, lq, body = (list(x) for x in zip(*reqs))
    n = max(-(-x // R) for x in kv)
    t = np.stack([np.roll(np.arange(n, dtype=np.int32), i) for i in range(len(kv))])      # (shared pages)
    pages = kvr.Pages(*(_randn(i, (n, 1, H, R, D), "bf16") for i in (1, 2)))
    kw = {}
    if any(body):
        packed = pool.packed_pages(n, R)
        pool.page_pack(pages, t[:1], packed, t[:1], [0], [max(body)])
        kw = dict(packed=packed, packed_table=t, packed_len=body)
    Q = _randn(3, (1, sum(lq), H * G, D), "bf16")
    want, out = torch.empty_like(Q), torch.zeros_like(Q)
    args = (pages, t, kv, _starts(lq).astype(np.int32), Q)
    pool.page_attention(*args, want, **kw)
    torch.cuda.synchronize()
    pool.check()
    gc.collect()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.add_(0)
        if fits:
            pool.page_attention(*args, out, **kw)
        else:
            with pytest.raises(kvr.KvrError) as e:
                pool.page_attention(*args, out, **kw)
            assert e.value.status == 3
    g.replay()
    torch.cuda.synchronize()
    pool.check()
    assert torch.equal(out, want) if fits else not out.any()


def test_a_padded_batch():
    """One layer: tokens behind the last request's are left as they were.  More layers: refused where the token
    axis is longer than the offsets, taken when cut to it."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    H, G, D, R = 2, 4, 128, 32
    for L in (1, 3):
        pool = _pool(L, H, G, D, "bf16")
        t, n = _table([90, 50], R, 3)
        pages = kvr.Pages(*(_randn(i, (n, L, H, R, D), "bf16") for i in (1, 2)))
        for lq in ((1, 1), (2, 3), (30, 9)):
            T, qo = sum(lq), _starts(lq).astype(np.int32)
            wide = _randn(3, (L, T + 5, H * G, D), "bf16")
            q, want, out = wide[:, :T].contiguous(), torch.empty_like(wide[:, :T]), torch.full_like(wide, 7.0)
            pool.page_attention(pages, t, [90, 50], qo, q, want)
            if L == 1:
                pool.page_attention(pages, t, [90, 50], qo, wide, out)
                torch.cuda.synchronize()
                assert torch.equal(out[:, :T], want) and (out[:, T:] == 7.0).all()
            else:
                for a, b in ((wide, out), (q, out), (wide, want.clone())):
                    with pytest.raises(ValueError, match="tokens in each layer"):
                        pool.page_attention(pages, t, [90, 50], qo, a, b)
            pool.check()
