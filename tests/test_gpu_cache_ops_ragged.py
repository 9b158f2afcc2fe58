"""Cache operators on batches of unlike requests, and where CTAs of a cluster
exchange results block after block.  References and tolerances are those of
test_gpu_cache_ops."""
import numpy as np
import pytest

from test_gpu_cache_ops import _pool, _randn, _shared_case, _starts, _weights_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,prefix", [([300, 200], [3000, 20]), ([64, 700, 1], [0, 1500, 9])])
def test_key_weights_of_many_row_blocks_in_a_cluster(q, prefix):
    """Three and more blocks of 128 query rows, a unit's tiles over a cluster of
    eight CTAs, most of which have no tile of the short request: the CTAs
    exchange their rows' sums block after block, hardly apart in time."""
    import torch
    _weights_case(1, 1, 4, 128, "bf16", prefix=prefix, q=q)
    pool, n = _pool(1, 1, 4, 128, "bf16"), len(q)
    co, qo = _starts([a + b for a, b in zip(prefix, q)]), _starts(q).astype(np.int32)
    ck, Q = _randn(1, (int(co[-1]), 128), "bf16"), _randn(2, (1, int(qo[-1]), 4, 128), "bf16")
    w = [torch.zeros(int(co[-1]), device="cuda") for _ in range(2)]
    pool.key_weights(co, prefix, qo, Q, ck, w[0])
    for _ in range(40):
        pool.key_weights(co, prefix, qo, Q, ck, w[1])
        assert torch.equal(w[0], w[1])
    # every query row's probabilities sum to one
    for b in range(n):
        got = float(w[0][int(co[b]):int(co[b + 1])].double().sum())
        assert abs(got - 4 * q[b]) <= 4 * q[b] * 2.0 ** -16


@pytest.mark.parametrize("groups,prefix,own,q", [([4], [2600], [100, 60, 33, 90], [1] * 4),
                                                  ([70], [900], [40] * 70, [1] * 70),
                                                  ([3, 2], [200, 385], [0, 3, 300, 128, 1], [100, 130, 33, 150, 99])])
def test_shared_prefix_behind_the_kernels_that_write_its_inputs(groups, prefix, own, q):
    """Prefix, own rows and queries written by kernels just before the call on its
    stream: the launches overlap at their ends, and every call reads this time's."""
    import torch
    L = 19 if sum(q) > 100 else 2
    pool, args, _ = _shared_case(L, 8, 4, 128, "bf16", groups=groups, prefix=prefix, own=own, q=q, check=())
    names = (3, 4, 8, 9, 10, 11, 12)
    out = args[-1]
    sets = []
    for k in range(3):
        x = [torch.randn_like(args[i]) for i in names]
        for i, y in zip(names, x):
            args[i].copy_(y)
        torch.cuda.synchronize()
        pool.shared_query_attention(*args)
        torch.cuda.synchronize()
        sets.append((x, out.clone()))
    got = []
    for k in range(30):
        x = sets[k % 3][0]
        for i, y in zip(names, x):
            args[i].copy_(y)
        pool.shared_query_attention(*args)
        got.append(out.clone())
    torch.cuda.synchronize()
    pool.check()
    for k, o in enumerate(got):
        assert torch.equal(o, sets[k % 3][1]), k


def test_shared_prefix_of_one_long_query_among_single_tokens():
    """A prefill in a batch of decode steps, requests without tokens between them."""
    q = [1] * 20 + [0, 300, 0, 0] + [1] * 10 + [130, 1, 0]
    own = [(7 * i) % 150 for i in range(len(q))]
    for L, H, G in ((1, 2, 4), (3, 1, 7)):
        _shared_case(L, H, G, 128, "bf16", groups=[22, len(q) - 22], prefix=[300, 129], own=own, q=q)
    n = 70   # a table in device memory
    _shared_case(1, 1, 4, 128, "bf16", groups=[n], prefix=[260], own=[i % 40 for i in range(n)], q=[1] * 33 + [170] + [1] * (n - 34))


def test_shared_prefix_grids_go_by_the_work():
    """Requests x the longest one's work (33,000 x 16,500 tokens x 64 units, by 16)
    is more CTAs than a grid holds; the work itself is small."""
    n, long = 33000, 16500
    q = [0] * n
    q[10], q[11], q[20000], q[32998] = 1, long, 2, 1
    _shared_case(8, 8, 1, 128, "bf16", groups=[n], prefix=[40], own=[0] * n, q=q, check=(10, 20000, 20001, 32998, 32999), spare=1)


def _us(fn):
    import torch
    t = []
    for k in range(8):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        torch.cuda._sleep(1000000)
        e[0].record()
        fn()
        e[1].record()
        torch.cuda.synchronize()
        if k > 2:
            t.append(1e3 * e[0].elapsed_time(e[1]))
    return sorted(t)[len(t) // 2]


def test_a_long_query_is_not_slower_for_the_single_tokens_beside_it():
    """A batch takes no more than three times what its parts take alone (one whose
    launches went by requests x the longest query took 27 times as long)."""
    def us(q, own):
        pool, args, _ = _shared_case(1, 8, 4, 128, "bf16", groups=[len(q)], prefix=[2592], own=own, q=q, check=())
        return _us(lambda: pool.shared_query_attention(*args))
    assert us([1] * 40 + [2048] + [1] * 23, [100] * 64) < 3 * (us([1] * 63, [100] * 63) + us([2048], [100]))


def test_key_weights_of_one_window_among_single_tokens():
    """Each request by the kernel for its own rows, whatever is beside it: the
    batch's order, requests without tokens, a table in device memory."""
    q = [1] * 5 + [0, 40, 8, 0, 200] + [1] * 6
    prefix = [(97 * i) % 700 for i in range(len(q))]
    for acc in (False, True):
        _weights_case(2, 1, 4, 128, "bf16", prefix=prefix, q=q, accumulate=acc)
    _weights_case(1, 2, 4, 128, "bf16", prefix=[30 + i for i in range(80)], q=[1] * 50 + [33] + [0] * 4 + [8] * 25)


def test_key_weights_of_single_tokens_beside_a_window():
    """Single tokens get the same weights bit for bit with and without a window in
    their batch (either way a CTA a unit, and three query terms), and the batch
    takes no longer than its parts."""
    import torch
    L, H, G, D, P = 8, 8, 4, 128, 1200
    pool = _pool(L, H, G, D, "bf16")

    def call(q):
        co, qo = _starts([P + n for n in q]), _starts(q).astype(np.int32)
        ck = _randn(1, (int(co[-1]) * L * H, D), "bf16", 2.0)
        Q = _randn(2, (L, int(qo[-1]), H * G, D), "bf16", 2.0)
        w = torch.empty(int(co[-1]) * L * H, device="cuda")
        return w, ck, Q, lambda: pool.key_weights(co, [P] * len(q), qo, Q, ck, w)

    w, ck, Q, run = call([1] * 6 + [64])
    w1, ck1, Q1, run1 = call([1] * 6)
    ck1.copy_(ck[:ck1.shape[0]])
    Q1.copy_(Q[:, :6])
    run()
    run1()
    torch.cuda.synchronize()
    pool.check()
    assert torch.equal(w[:w1.numel()], w1)
    single, window, both = (_us(call(q)[3]) for q in ([1] * 63, [2048], [1] * 40 + [2048] + [1] * 23))
    assert both < 1.5 * (single + window)


@pytest.mark.parametrize("D,dtype", [(64, "fp32"), (128, "bf16")])
def test_reserved_pool_takes_every_request_table(D, dtype):
    """After kvr_pool_reserve no call within the limits waits for the GPU: each
    returns while a kernel enqueued before it still runs."""
    import torch
    B, L, H, G = 1000, 1, 1, 2
    pool = _pool(L, H, G, D, dtype)
    pool.reserve(max_batch=B, max_query_tokens=B)
    co, qo = np.arange(B + 1) * 6, np.arange(B + 1)
    ck, cv = _randn(1, (6 * B, D), dtype), _randn(2, (6 * B, D), dtype)
    q, kq, vq = _randn(3, (L, B, H * G, D), dtype), _randn(4, (L, B, H, D), dtype), _randn(5, (L, B, H, D), dtype)
    out, w = torch.empty_like(q), torch.zeros(6 * B, device="cuda")
    kept, own = torch.empty(2 * B, device="cuda", dtype=torch.int32), [3] * B

    def calls(n):
        c, o, t = co[:n + 1], own[:n], qo[:n + 1]
        x = [y[:, :n].contiguous() for y in (q, kq, vq, out)]
        # (a group of each request, nothing shared: no partial results)
        yield lambda: pool.shared_query_attention(t, [0] * (n + 1), [0] * n, None, None, c, o, t, *x[:3], ck, cv, x[3])
        yield lambda: pool.key_weights(c, o, t, x[0], ck, w)
        yield lambda: pool.evict(c, [4] * n, [2] * n, w, ck, cv, kept)

    for call in calls(3):     # (kernels are loaded)
        call()
    for call in calls(B):
        for _ in range(3):
            torch.cuda.synchronize()
            torch.cuda._sleep(600_000_000)
            done = torch.cuda.Event()
            done.record()
            call()
            assert not done.query()
    torch.cuda.synchronize()
    pool.check()


@pytest.mark.parametrize("D,dtype", [(64, "fp32"), (128, "bf16")])
def test_shared_prefix_writes_the_output_over_the_queries(D, dtype):
    import torch
    pool, args, (ck0, cv0) = _shared_case(2, 2, 4, D, dtype, groups=[3], prefix=[300], own=[5, 40, 0], q=[1, 30, 2])
    want, q = args[-1].clone(), args[8].clone()
    pool.shared_query_attention(*args[:8], q, *args[9:-1], q)
    torch.cuda.synchronize()
    pool.check()
    assert torch.equal(q, want)


def test_key_weights_of_the_longest_cache_and_many_heads():
    """2^24 rows, 130 query heads on one kv head: row numbers times heads pass 32
    bits.  Every key weighs the same: 130 / 2^24, which fp32 holds exactly."""
    import torch
    n, G, D = 1 << 24, 130, 64
    pool = _pool(1, 1, G, D, "bf16")
    ck = torch.zeros((n, D), device="cuda", dtype=torch.bfloat16)
    q, w = _randn(1, (1, 1, G, D), "bf16"), torch.empty(n, device="cuda")
    pool.key_weights([0, n], [n - 1], [0, 1], q, ck, w)
    torch.cuda.synchronize()
    pool.check()
    assert (w == G / n).all()


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("q,prefix", [([12], [900]), ([60, 40], [2500, 300]), ([90], [700])])
def test_key_weights_of_a_window_with_growing_and_falling_scores(q, prefix, up):
    """More than 32 (and 128) query rows, keys of growing (falling) length: the
    rows' references move in every tile, or never again.

    Elementwise the bound of the other tests.  In the 2-norm: a score is off by the
    query bits that two bf16 terms leave (independent, 2^-18 / sqrt 3 each: 17.3 *
    2^-18 / sqrt 3 = 3.8e-5 for the longest keys' scores of deviation 17.3) and by 128
    fp32 additions to sums of up to 64 (sqrt(128) * 64 * 2^-24 = 4.3e-5); numerator
    and denominator: 1.2e-4, 2^-13."""
    import oracle
    import torch
    from parity import to_np64
    from test_gpu_cache_ops import THETA, _attention_ref, _block
    L, H, G, D = 1, 2, 4, 128
    B, LH, T = len(q), L * H, sum(q)
    co, qo = _starts([a + b + 3 for a, b in zip(prefix, q)]), _starts(q).astype(np.int32)
    ck = _randn(1, (int(co[-1]) * LH, D), "bf16", 1.7)
    Q = _randn(2, (L, T, H * G, D), "bf16", 1.7)
    for b in range(B):
        blk = _block(ck, co, b, LH)
        f = torch.linspace(0.01, 6.0, prefix[b] + q[b], device="cuda")
        blk[:, :len(f)] *= (f if up else f.flip(0))[None, :, None].to(blk.dtype)
        blk[:, len(f):] = float("nan")
    pool, w = _pool(L, H, G, D, "bf16"), torch.full((int(co[-1]) * LH,), -1.0, device="cuda")
    pool.key_weights(co, prefix, qo, Q, ck, w)
    torch.cuda.synchronize()
    pool.check()
    e2 = n2 = 0.0
    for b in range(B):
        P, lq, a = prefix[b], q[b], int(qo[b])
        n, sc = P + lq, D ** -0.5
        got, K = to_np64(_block(w, co, b, LH)), to_np64(_block(ck, co, b, LH))
        assert (got[:, n:] == -1).all()
        qr = oracle.rope(to_np64(Q[:, a:a + lq]), P + np.arange(lq, dtype=np.float64)[None, :, None], THETA, False)
        for u in range(LH):
            _, _, qk, p = _attention_ref(K[u, :n], np.zeros((n, 1)), qr[0, :, u * G:(u + 1) * G], 0, P, sc)
            d = qk.max(-1) * (2.0 ** -16 + (D + 8) * 2.0 ** -24)
            ref = p.sum((0, 1))
            bound = (p * (np.exp(2 * d)[..., None] * (1 + n * 2.0 ** -23) - 1)).sum((0, 1)) + (lq * G + 2) * 2.0 ** -24 * ref + 1e-37
            err = np.abs(got[u, :n] - ref)
            assert (err <= bound).all(), (b, u, float((err / bound).max()))
            e2, n2 = e2 + (err ** 2).sum(), n2 + (ref ** 2).sum()
    assert (e2 / n2) ** 0.5 <= 2.0 ** -13, (e2 / n2) ** 0.5


# what the cases of test_gpu_cache_ops.WHOLE run, whose blocks of one row are not well filled
WHOLE_PATHS = {"two-groups": 2, "odd-heads": 2, "some-without-tokens": 2, "many-requests": 2, "one-row-blocks": 1}


@pytest.mark.parametrize("name", WHOLE_PATHS)
def test_which_kernels_the_cases_of_many_query_blocks_run(name):
    from test_gpu_cache_ops import WHOLE
    assert set(WHOLE) == set(WHOLE_PATHS)
    c = dict(WHOLE[name])
    pool = _shared_case(c.pop("L"), 8, c.pop("G"), 128, "bf16", check=(), **c)[0]
    assert pool.shared_path == WHOLE_PATHS[name]


def test_which_kernels_short_queries_run():
    kw = dict(groups=[2], prefix=[100], own=[3, 4], check=())
    assert _shared_case(1, 2, 2, 64, "fp32", q=[1, 1], **kw)[0].shared_path == 0
    assert _shared_case(1, 2, 2, 128, "bf16", q=[1, 9], **kw)[0].shared_path == 1


@pytest.mark.parametrize("own_scale", [0.02, 8.0])
def test_shared_prefix_whole_blocks_with_moving_maxima(own_scale):
    """Whole blocks of query rows whose prefix keys grow, and whose own keys are
    far longer (a row's maximum moves in an own tile, which only some rows of a warp
    see) or far shorter, against query attention on prefix and own rows in one cache.

    Both round the same rotated queries and keys and each probability once, to a
    reference of their own: with A = sum_j p_j |v_j| each is off by its output's
    rounding, its probabilities' and n fp32 additions: 2 (2^-8 A + 2^-8 A + n 2^-23 A)
    apart.  A comes from the rounded inputs, within 2^-7 of itself."""
    import oracle
    import torch
    from parity import to_np64
    from test_gpu_cache_ops import THETA, _attention_ref, _block
    L, H, G, D, P, own, q = 19, 8, 4, 128, 200, [130, 60], [100, 130]
    LH = L * H
    pool, args, (ck0, cv0) = _shared_case(L, H, G, D, "bf16", groups=[2], prefix=[P], own=own, q=q, check=())
    go, po, _, pk, pv, co, _, qo, Q, KQ, VQ, ck, cv, out = args
    pk, kq = pk.clone(), KQ * own_scale
    _block(pk, po, 0, LH)[:, :P] *= torch.linspace(0.05, 4.0, P, device="cuda")[None, :, None].to(pk.dtype)
    ck.copy_(ck0)
    for b in range(2):
        _block(ck, co, b, LH)[:, :own[b]] *= own_scale
    fo = _starts([P + a + b for a, b in zip(own, q)])
    fk, fv = (torch.zeros((int(fo[-1]) * LH, D), device="cuda", dtype=ck.dtype) for _ in range(2))
    for b in range(2):
        for f, p, o in ((fk, pk, ck), (fv, pv, cv0)):
            blk = _block(f, fo, b, LH)
            blk[:, :P], blk[:, P:P + own[b]] = _block(p, po, 0, LH)[:, :P], _block(o, co, b, LH)[:, :own[b]]
    pool.shared_query_attention(go, po, [P], pk, pv, co, own, qo, Q, kq, VQ, ck, cv, out)
    assert pool.shared_path == 2
    want = torch.empty_like(out)
    pool.query_attention(fo, [P + a for a in own], qo, Q, kq, VQ, fk, fv, want)
    torch.cuda.synchronize()
    pool.check()
    for b in range(2):
        a, n = int(qo[b]), P + own[b] + q[b]
        pos = P + own[b] + np.arange(q[b], dtype=np.float64)
        qr = to_np64(torch.from_numpy(oracle.rope(to_np64(Q[:, a:a + q[b]]), pos[None, :, None], THETA, False)).to(Q.dtype))
        K, V = to_np64(_block(fk, fo, b, LH)), to_np64(_block(fv, fo, b, LH))
        x, y = to_np64(out[:, a:a + q[b]]), to_np64(want[:, a:a + q[b]])
        for u in range(0, LH, 5):
            l, h = divmod(u, H)
            hs = slice(h * G, (h + 1) * G)
            _, A, _, _ = _attention_ref(K[u], V[u], qr[l, :, hs], 0, P + own[b], D ** -0.5)
            err = np.abs(x[l, :, hs] - y[l, :, hs])
            bound = 2 * (2 * 2.0 ** -8 + n * 2.0 ** -23) * A * (1 + 2.0 ** -7)
            assert (err <= bound).all(), (b, u, float((err / bound).max()))
