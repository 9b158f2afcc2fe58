"""Paged cache: what a call uses beside its arguments."""
import threading

import pytest

from test_gpu_page_cache import _pool, _randn, _table

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
