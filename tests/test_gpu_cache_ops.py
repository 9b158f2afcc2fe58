"""Shared-prefix attention, key weights and eviction on the GPU against plain
fp64 numpy (rotations and attention of the oracle).

Tolerances, in half steps u of a type (bf16 2^-8, fp32 2^-24) relative to a
value:
* attention output: with A = sum_j p_j |v_j| and d = the largest change that
  rounding the row's query and one key can make to a score,
      |o - o_ref| <= u |o_ref| + A ((1 + u) e^{2d} - 1) + n 2^-23 A:
  the output is rounded once, each probability once (to bf16 on the tensor
  cores), and a score off by at most d moves p by a factor within e^{+-2d}
  (numerator and denominator).  In bf16 d = scale sum_i |q_i k_i| 2u (query
  and appended key rounded); in fp32, with D products and a rotation of 4
  roundings each way, d = scale sum_i |q_i k_i| (D + 8) u.  In the 2-norm the
  three roundings are independent and add in squares: ||o - o_ref|| <= sqrt(3)
  2^-8 ||o_ref|| in bf16; in fp32, scores off by up to 2^-17, 2^-17 ||o_ref||.
* weights: queries keep 16 bits (2^-16 relative) and sums are fp32, so
  d = scale sum_i |q_i k_i| (2^-16 + (D + 8) 2^-24), and each row's part of a
  weight is off by at most (e^{2d} (1 + n 2^-23) - 1) of itself; in the 2-norm,
  where the bits of queries and products are independent, 2^-16.
* kept rows, moved values and weights: exact.  Moved keys: the stitched keys'
  tolerance (two steps of a bf16; 2^-20 of the pair's norm in fp32).
"""
import numpy as np
import pytest

import oracle
from parity import k_within_tolerance, to_np64

pytestmark = pytest.mark.gpu

THETA = 1e6


def _dt(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _pool(L, H, G, D, dtype, il=False, theta=THETA):
    import torch
    from rag_precomputed_kv_gb300 import kvr
    k = torch.zeros((1, L, H, 8, D), device="cuda", dtype=_dt(dtype))
    return kvr.Pool(k, torch.zeros_like(k), H * G, theta, rope_interleaved=il)


def _randn(seed, shape, dtype, scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(_dt(dtype))


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _block(flat, offsets, b, LH):
    """Request b's block [LH, R_b, ...] of a flat cache."""
    return flat[int(offsets[b]) * LH:int(offsets[b + 1]) * LH].reshape((LH, int(offsets[b + 1] - offsets[b])) + tuple(flat.shape[1:]))


def _attention_ref(K, V, q, first_pos, n_own_before, scale):
    """K, V [n, D] fp64; q [Lq, G, D] rotated; token t sees rows < n_own_before + t + 1.
    Returns o, and per output the bound's ingredients A and sum |q k| (max over keys)."""
    Lq, G, n = q.shape[0], q.shape[1], K.shape[0]
    rows = lambda x, y: (x.reshape(Lq * G, -1) @ y).reshape(Lq, G, -1)
    s = rows(q, K.T) * scale
    vis = np.arange(n)[None, :] <= n_own_before + np.arange(Lq)[:, None]
    s = np.where(vis[:, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    qk = np.where(vis[:, None], rows(np.abs(q), np.abs(K).T), 0.0) * scale
    return rows(p, V), rows(p, np.abs(V)), qk, p


def _check_attention(got, ref, A, qk, n, dtype, D):
    if dtype == "bf16":
        u = 2.0 ** -8
        d = qk.max(-1) * 2 * u
        p_round = 1 + u
    else:
        u = 2.0 ** -24
        d = qk.max(-1) * (D + 8) * u
        p_round = 1.0
    bound = u * np.abs(ref) + A * (p_round * np.exp(2 * d)[..., None] - 1) + n * 2.0 ** -23 * A
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= bound).all(), float((err / bound).max())
    return float((err ** 2).sum()), float((ref ** 2).sum())


# ---------------------------------------------------------------------------
# shared prefix
# ---------------------------------------------------------------------------
def _shared_case(L, H, G, D, dtype, groups, prefix, own, q, il=False, theta=THETA, scale=0.0, seed=1, spread=1.0,
                 stream=None, spare=3, pool=None, check=None):
    """groups: requests per group; prefix per group; own and q per request.
    check: the requests whose results are compared (None: all)."""
    import torch
    B, LH, T = sum(groups), L * H, int(sum(q))
    go, po = _starts(groups).astype(np.int32), _starts([p + 2 for p in prefix])
    co, qo = _starts([a + b + spare for a, b in zip(own, q)]), _starts(q).astype(np.int32)
    pk, pv = (_randn(seed + i, (int(po[-1]) * LH, D), dtype, spread) for i in (0, 1))
    ck, cv = (_randn(seed + i, (int(co[-1]) * LH, D), dtype, spread) for i in (2, 3))
    Q, KQ, VQ = (_randn(seed + 4, (L, T, H * G, D), dtype, spread), _randn(seed + 5, (L, T, H, D), dtype, spread),
                 _randn(seed + 6, (L, T, H, D), dtype, spread))
    # rows that hold no data are NaN: nothing may come of them
    for g, P in enumerate(prefix):
        for x in (pk, pv):
            _block(x, po, g, LH)[:, P:] = float("nan")
    for b in range(B):
        for x in (ck, cv):
            _block(x, co, b, LH)[:, own[b]:] = float("nan")
    pool = pool or _pool(L, H, G, D, dtype, il, theta)
    out = torch.full_like(Q, float("nan"))
    ck0, cv0, pk0, pv0 = ck.clone(), cv.clone(), pk.clone(), pv.clone()
    torch.cuda.synchronize()
    args = (go, po, prefix, pk, pv, co, own, qo, Q, KQ, VQ, ck, cv, out)
    pool.shared_query_attention(*args, softmax_scale=scale, stream=stream)
    torch.cuda.synchronize()
    pool.check()
    sc = scale if scale > 0 else D ** -0.5
    e2 = n2 = 0.0
    for g in range(len(groups)):
        Kp, Vp = (to_np64(_block(x, po, g, LH))[:, :prefix[g]] for x in (pk, pv))
        for b in range(int(go[g]), int(go[g + 1])):
            if check is not None and b not in check:
                continue
            S, lq, a = own[b], q[b], int(qo[b])
            gk, gv = to_np64(_block(ck, co, b, LH)), to_np64(_block(cv, co, b, LH))
            wk, wv = to_np64(_block(ck0, co, b, LH)), to_np64(_block(cv0, co, b, LH))
            assert np.array_equal(gk[:, :S], wk[:, :S]) and np.array_equal(gv[:, :S], wv[:, :S])
            assert np.isnan(gk[:, S + lq:]).all() and np.isnan(gv[:, S + lq:]).all()   # left as they were
            if lq == 0:
                continue
            pos = prefix[g] + S + np.arange(lq, dtype=np.float64)
            kq, vq = to_np64(KQ[:, a:a + lq]), to_np64(VQ[:, a:a + lq])
            kr = oracle.rope(np.moveaxis(kq, 2, 1).reshape(LH, lq, D), pos[None, :], theta, il)
            assert k_within_tolerance(gk[:, S:S + lq], kr, dtype, il)[0]
            assert np.array_equal(gv[:, S:S + lq], np.moveaxis(vq, 2, 1).reshape(LH, lq, D))
            qr, outn = oracle.rope(to_np64(Q[:, a:a + lq]), pos[None, :, None], theta, il), to_np64(out[:, a:a + lq])
            for u in range(LH):
                l, h = divmod(u, H)
                K = np.concatenate([Kp[u], gk[u, :S], kr[u]])
                V = np.concatenate([Vp[u], gv[u, :S + lq]])
                ref, A, qk, _ = _attention_ref(K, V, qr[l, :, h * G:(h + 1) * G], 0, prefix[g] + S, sc)
                x, y = _check_attention(outn[l, :, h * G:(h + 1) * G], ref, A, qk, len(K), dtype, D)
                e2, n2 = e2 + x, n2 + y
    rel = (e2 / max(n2, 1e-300)) ** 0.5
    assert rel <= (3 ** 0.5 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17), rel
    for x, y in ((pk, pk0), (pv, pv0)):
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))
    return pool, args, (ck0, cv0)


SHARED = {
    "one-request-one-key": dict(groups=[1], prefix=[0], own=[0], q=[1]),
    "one-prefix-row": dict(groups=[1], prefix=[1], own=[0], q=[1]),
    "decode": dict(groups=[3], prefix=[131], own=[5, 0, 17], q=[1, 1, 1]),
    "tile-edges": dict(groups=[2, 1, 1], prefix=[128, 127, 129], own=[127, 128, 1, 200], q=[1, 1, 1, 1]),
    "some-without-tokens": dict(groups=[3, 2], prefix=[70, 300], own=[5, 2, 17, 9, 0], q=[1, 0, 1, 0, 1]),
    "empty-groups": dict(groups=[0, 2, 0, 1], prefix=[9, 257, 0, 40], own=[3, 4, 5], q=[1, 2, 1]),
    "nothing-shared": dict(groups=[2], prefix=[0], own=[140, 3], q=[1, 9]),
    "queries": dict(groups=[2, 2], prefix=[200, 385], own=[0, 3, 130, 0], q=[7, 33, 1, 64]),
    "short-queries": dict(groups=[12, 9], prefix=[700, 260], own=[7 * i % 40 for i in range(21)], q=[5 + i % 4 for i in range(21)]),
    "short-queries-long-own": dict(groups=[5], prefix=[700], own=[260, 0, 391, 127, 128], q=[9, 5, 8, 12, 7]),
    "long-queries": dict(groups=[2], prefix=[150], own=[0, 40], q=[150, 271]),
    "many": dict(groups=[40, 30], prefix=[140, 64], own=[i % 7 for i in range(70)], q=[1 + (i % 5 == 0) for i in range(70)]),
}


@pytest.mark.parametrize("name", SHARED)
@pytest.mark.parametrize("L,H,G,D,dtype", [(2, 2, 4, 128, "bf16"), (1, 2, 2, 64, "fp32"), (1, 1, 3, 64, "bf16"),
                                            (1, 1, 2, 128, "fp32")])
def test_shared_prefix(name, L, H, G, D, dtype):
    _shared_case(L, H, G, D, dtype, **SHARED[name])


@pytest.mark.parametrize("G", [1, 2, 7, 8, 16, 20])
def test_shared_prefix_group_sizes(G):
    _shared_case(1, 2, G, 128, "bf16", groups=[5], prefix=[333], own=[0, 1, 20, 128, 131], q=[1, 3, 1, 1, 2])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 64)])
def test_shared_prefix_interleaved_pairs_far_positions_and_scale(dtype, D):
    _shared_case(1, 2, 4, D, dtype, groups=[2], prefix=[4500], own=[3, 9], q=[1, 2], il=True, theta=1e4, scale=0.03)


@pytest.mark.parametrize("rows", [127, 128, 129, 255, 256, 257, 513])
def test_shared_prefix_query_rows_at_tile_edges(rows):
    """All requests of a group in one (layer, kv-head)'s query rows: G = 1."""
    _shared_case(1, 1, 1, 128, "bf16", groups=[rows], prefix=[260], own=[i % 3 for i in range(rows)], q=[1] * rows)


# enough blocks of 256 query rows for every SM: prefix and own keys in one kernel
WHOLE = {
    "two-groups": dict(G=4, L=19, groups=[3, 2], prefix=[200, 385], own=[0, 3, 300, 128, 1], q=[100, 130, 33, 150, 99]),
    "odd-heads": dict(G=7, L=16, groups=[1, 3], prefix=[1, 129], own=[127, 0, 40, 5], q=[128, 64, 1, 190]),
    "some-without-tokens": dict(G=16, L=19, groups=[2, 0, 3], prefix=[64, 9, 128], own=[7, 2, 0, 9, 129], q=[150, 0, 0, 127, 1]),
    "many-requests": dict(G=8, L=2, groups=[40, 30], prefix=[140, 385], own=[i % 7 for i in range(70)],
                          q=[20 + i % 5 for i in range(70)]),
    "one-row-blocks": dict(G=1, L=24, groups=[1] * 8, prefix=[300 + i for i in range(8)], own=list(range(8)), q=[1] * 8),
}


@pytest.mark.parametrize("name", WHOLE)
def test_shared_prefix_of_many_query_blocks(name):
    c = dict(WHOLE[name])
    L, G = c.pop("L"), c.pop("G")
    _shared_case(L, 8, G, 128, "bf16", **c)


@pytest.mark.parametrize("q", [[1, 1], [3, 1]])
def test_shared_prefix_of_more_heads_than_a_tile_has_rows(q):
    _shared_case(1, 1, 130, 128, "bf16", groups=[2], prefix=[300], own=[0, 70], q=q)


def test_shared_prefix_of_many_query_blocks_keeps_requests_apart():
    """What is not a number in one request's values and keys reaches none of the
    others, which share its blocks of query rows."""
    import torch
    q = [100, 30, 70, 33, 200, 79]
    pool, args, _ = _shared_case(19, 8, 4, 128, "bf16", groups=[6], prefix=[200], own=[5, 0, 9, 130, 1, 2], q=q, check=(1,))
    want = args[-1].clone()
    qo = _starts(q)
    a, b = int(qo[2]), int(qo[3])
    args[9][:, a + 3:b, :, 5] = float("nan")
    args[10][:, a:b, :, ::3] = float("inf")
    args[10][:, a:b, :, 1] = float("nan")
    pool.shared_query_attention(*args)
    torch.cuda.synchronize()
    got = args[-1]
    for x, y in ((0, a), (b, int(qo[-1]))):
        assert torch.equal(got[:, x:y], want[:, x:y])
    assert not torch.isfinite(got[:, a:b]).all()


def test_shared_prefix_in_slices():
    """More than 1 GiB of partial results (64 units x 128 blocks of 256 rows):
    the units go through in two slices."""
    n = 4096
    _shared_case(8, 8, 8, 128, "bf16", groups=[n], prefix=[130], own=[i % 3 for i in range(n)], q=[1] * n,
                 check=(0, 1, 1500, 2047, 4095))


def test_shared_prefix_large_scores():
    """Scores of some hundreds, the largest keys late: the running maximum moves."""
    import torch
    L, H, G, D, P = 1, 2, 4, 128, 700
    pool = _pool(L, H, G, D, "bf16")
    K = _randn(1, (P * H, D), "bf16", 0.02).view(H, P, D)
    V = _randn(2, (P * H, D), "bf16").view(H, P, D)
    q = _randn(3, (L, 2, H * G, D), "bf16", 0.5)
    # the rotation at position P + 0 is undone, so that key j points along the query
    qr = oracle.rope(to_np64(q), np.full((1, 2, 1), float(P)), THETA)
    for j, a in ((0, 1.0), (130, 4.0), (300, 9.0), (555, 16.0), (699, 12.0)):
        for h in range(H):
            K[h, j] = torch.from_numpy(qr[0, 0, h * G] * a).to(K)
    ck = torch.full((2 * H * 2, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    cv = ck.clone()
    kq, vq = _randn(4, (L, 2, H, D), "bf16"), _randn(5, (L, 2, H, D), "bf16")
    out = torch.empty_like(q)
    pool.shared_query_attention([0, 2], [0, P], [P], K.reshape(-1, D), V.reshape(-1, D), [0, 2, 4], [0, 0], [0, 1, 2],
                                q, kq, vq, ck, cv, out)
    torch.cuda.synchronize()
    pool.check()
    kr = oracle.rope(to_np64(kq), np.full((1, 2, 1), float(P)), THETA)
    for b in range(2):
        for h in range(H):
            Kf = np.concatenate([to_np64(K[h]), kr[0, b, h][None]])
            Vf = np.concatenate([to_np64(V[h]), to_np64(vq[0, b, h])[None]])
            ref, A, qk, _ = _attention_ref(Kf, Vf, qr[:, b, h * G:(h + 1) * G], 0, P, D ** -0.5)
            _check_attention(to_np64(out[:, b, h * G:(h + 1) * G]), ref, A, qk, P + 1, "bf16", D)


@pytest.mark.parametrize("rows", [24, 200])
def test_shared_prefix_of_growing_scores(rows):
    """Prefix keys of growing length: every row's maximum moves, at tiles of its own."""
    import torch
    L, H, G, D, P, B = 1, 2, 4, 128, 900, rows // 4
    pool = _pool(L, H, G, D, "bf16")
    K, V = _randn(1, (H, P, D), "bf16"), _randn(2, (H, P, D), "bf16")
    K = (K.float() * torch.linspace(0.05, 6.0, P, device="cuda")[None, :, None]).to(K.dtype)
    q, kq, vq = _randn(3, (L, B, H * G, D), "bf16"), _randn(4, (L, B, H, D), "bf16"), _randn(5, (L, B, H, D), "bf16")
    ck = torch.full((B * H * 2, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    cv, out = ck.clone(), torch.empty_like(q)
    pool.shared_query_attention([0, B], [0, P], [P], K.reshape(-1, D), V.reshape(-1, D), np.arange(B + 1) * 2, [0] * B,
                                np.arange(B + 1), q, kq, vq, ck, cv, out)
    torch.cuda.synchronize()
    pool.check()
    pos = np.full((1, 1, 1), float(P))
    qr, kr = oracle.rope(to_np64(q), pos, THETA), oracle.rope(to_np64(kq), pos, THETA)
    for b in range(B):
        for h in range(H):
            Kf = np.concatenate([to_np64(K[h]), kr[0, b, h][None]])
            Vf = np.concatenate([to_np64(V[h]), to_np64(vq[0, b, h])[None]])
            ref, A, qk, _ = _attention_ref(Kf, Vf, qr[:, b, h * G:(h + 1) * G], 0, P, D ** -0.5)
            _check_attention(to_np64(out[:, b, h * G:(h + 1) * G]), ref, A, qk, P + 1, "bf16", D)


def test_query_attention_of_growing_scores():
    """The same through the query prefill on a cache of its own."""
    import torch
    L, H, G, D, P, B, lq = 1, 2, 4, 128, 900, 2, 20
    pool, R = _pool(L, H, G, D, "bf16"), 930
    ck, cv = _randn(1, (B * H * R, D), "bf16"), _randn(2, (B * H * R, D), "bf16")
    scale = torch.cat([torch.linspace(0.05, 6.0, P, device="cuda"), torch.zeros(R - P, device="cuda")])
    ck = (ck.float().view(B * H, R, D) * scale[None, :, None]).to(ck.dtype).view(-1, D)
    q, kq, vq = _randn(3, (L, B * lq, H * G, D), "bf16"), _randn(4, (L, B * lq, H, D), "bf16"), _randn(5, (L, B * lq, H, D), "bf16")
    out = torch.empty_like(q)
    pool.query_attention(np.arange(B + 1) * R, [P] * B, np.arange(B + 1) * lq, q, kq, vq, ck, cv, out)
    torch.cuda.synchronize()
    pool.check()
    pos = P + np.arange(lq, dtype=np.float64)
    for b in range(B):
        sl = slice(b * lq, (b + 1) * lq)
        qr = oracle.rope(to_np64(q[:, sl]), pos[None, :, None], THETA)
        kr = oracle.rope(to_np64(kq[:, sl]), pos[None, :, None], THETA)
        for h in range(H):
            blk = slice((b * H + h) * R, (b * H + h) * R + P)
            K = np.concatenate([to_np64(ck[blk]), kr[0, :, h]])
            V = np.concatenate([to_np64(cv[blk]), to_np64(vq[0, sl, h])])
            ref, A, qk, _ = _attention_ref(K, V, qr[0, :, h * G:(h + 1) * G], 0, P, D ** -0.5)
            _check_attention(to_np64(out[0, sl, h * G:(h + 1) * G]), ref, A, qk, len(K), "bf16", D)


def test_shared_prefix_flags_bad_input():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    for dtype, D in (("bf16", 128), ("fp32", 64)):
        pool, args, _ = _shared_case(1, 2, 2, D, dtype, groups=[2], prefix=[140], own=[3, 0], q=[1, 1])
        args[8][0, 1, 1, 5] = float("nan")
        pool.shared_query_attention(*args)
        with pytest.raises(kvr.KvrError) as e:
            pool.check()
        assert e.value.status == 6
        pool.check()
        out = args[-1]
        assert torch.isfinite(out[0, 0]).all() and torch.isfinite(out[0, 1, 2:]).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 64)])
def test_shared_prefix_repeats_bit_for_bit_on_two_streams(dtype, D):
    """One pool used from two streams, its scratch shared: each call's result
    is the one it has alone."""
    import torch
    kw = dict(groups=[5], prefix=[700], own=[3, 0, 9, 2, 140], q=[1, 1, 1, 1, 2])
    pool, args, _ = _shared_case(2, 2, 4, D, dtype, **kw)
    pool, args2, _ = _shared_case(2, 2, 4, D, dtype, seed=31, pool=pool, **kw)
    want, want2 = args[-1].clone(), args2[-1].clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        pool.shared_query_attention(*args, stream=s1)
        pool.shared_query_attention(*args2, stream=s2)
    torch.cuda.synchronize()
    pool.check()
    assert torch.equal(args[-1], want) and torch.equal(args2[-1], want2)


# ---------------------------------------------------------------------------
# key weights
# ---------------------------------------------------------------------------
def _weights_case(L, H, G, D, dtype, prefix, q, il=False, theta=THETA, scale=0.0, accumulate=False, seed=1, spread=1.0,
                  spare=4, edit=None):
    import torch
    B, LH, T = len(prefix), L * H, int(sum(q))
    co, qo = _starts([a + b + spare for a, b in zip(prefix, q)]), _starts(q).astype(np.int32)
    ck = _randn(seed, (int(co[-1]) * LH, D), dtype, spread)
    Q = _randn(seed + 1, (L, max(T, 1), H * G, D), dtype, spread)[:, :T].contiguous()
    w = torch.rand(int(co[-1]) * LH, device="cuda")
    for b in range(B):
        _block(ck, co, b, LH)[:, prefix[b] + q[b]:] = float("nan")
    if edit:
        edit(ck, Q, co)
    pool = _pool(L, H, G, D, dtype, il, theta)
    w0 = w.clone()
    torch.cuda.synchronize()
    pool.key_weights(co, prefix, qo, Q if T else None, ck, w, softmax_scale=scale, accumulate=accumulate)
    torch.cuda.synchronize()
    pool.check()
    sc = scale if scale > 0 else D ** -0.5
    e2 = n2 = 0.0
    for b in range(B):
        P, lq, a = prefix[b], q[b], int(qo[b])
        n = P + lq
        got, old, K = to_np64(_block(w, co, b, LH)), to_np64(_block(w0, co, b, LH)), to_np64(_block(ck, co, b, LH))
        assert np.array_equal(got[:, n:], old[:, n:])
        base = old[:, :n] if accumulate else np.zeros((LH, n))
        if lq == 0:
            assert np.array_equal(got[:, :n], base)
            continue
        qr = oracle.rope(to_np64(Q[:, a:a + lq]), P + np.arange(lq, dtype=np.float64)[None, :, None], theta, il)
        for u in range(LH):
            l, h = divmod(u, H)
            _, _, qk, p = _attention_ref(K[u, :n], np.zeros((n, 1)), qr[l, :, h * G:(h + 1) * G], 0, P, sc)
            d = qk.max(-1) * (2.0 ** -16 + (D + 8) * 2.0 ** -24)
            part = p * (np.exp(2 * d)[..., None] * (1 + n * 2.0 ** -23) - 1)
            ref = base[u] + p.sum((0, 1))
            # the sum of Lq * G parts and the addition to what is there
            bound = part.sum((0, 1)) + (lq * G + 2) * 2.0 ** -24 * ref + 1e-37
            err = np.abs(got[u, :n] - ref)
            assert (err <= bound).all(), (b, u, float((err / bound).max()))
            e2, n2 = e2 + (err ** 2).sum(), n2 + (ref ** 2).sum()
    assert (e2 / max(n2, 1e-300)) ** 0.5 <= 2.0 ** -16
    return pool


WEIGHTS = {
    "one-key": dict(prefix=[0], q=[1]),
    "decode": dict(prefix=[300], q=[1]),
    "tile-edges": dict(prefix=[126, 127, 128, 129, 255], q=[1, 1, 1, 1, 1]),
    "window": dict(prefix=[200, 0, 77], q=[16, 33, 1]),
    "no-prefix": dict(prefix=[0, 0], q=[130, 7]),
    "some-without-tokens": dict(prefix=[40, 0, 30, 129], q=[0, 0, 3, 0]),
    "long": dict(prefix=[5000, 900], q=[1, 2]),
    "long-window": dict(prefix=[2100], q=[40]),
    "many": dict(prefix=[20 + i for i in range(70)], q=[1 + i % 3 for i in range(70)]),
}


@pytest.mark.parametrize("name", WEIGHTS)
@pytest.mark.parametrize("L,H,G,D,dtype", [(2, 2, 4, 128, "bf16"), (1, 2, 2, 64, "fp32"), (1, 1, 3, 64, "bf16"),
                                            (1, 1, 2, 128, "fp32")])
def test_key_weights(name, L, H, G, D, dtype):
    _weights_case(L, H, G, D, dtype, **WEIGHTS[name], accumulate=name in ("decode", "long", "some-without-tokens"))


@pytest.mark.parametrize("G", [1, 7, 8, 16, 17, 32, 130])
@pytest.mark.parametrize("q", [1, 5, 40])
def test_key_weights_group_sizes(G, q):
    _weights_case(1, 1, G, 128, "bf16", prefix=[333, 1500], q=[q, 1], accumulate=q == 5)


@pytest.mark.parametrize("G,q,n", [(4, 1, 50000), (8, 1, 25500), (16, 1, 11000), (16, 2, 6200), (32, 1, 6000)])
def test_key_weights_of_more_keys_than_tmem_holds(G, q, n):
    """The tiles beyond what eight CTAs keep (6,144 keys each at up to 4 rows,
    down to 640 at 32) are loaded twice; a second, short request beside it."""
    _weights_case(1, 1, G, 128, "bf16", prefix=[n - q, 40], q=[q, 1], accumulate=G == 8)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 64)])
def test_key_weights_interleaved_pairs_far_positions_and_scale(dtype, D):
    _weights_case(1, 2, 4, D, dtype, prefix=[4500], q=[9], il=True, theta=1e4, scale=0.05)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("up", [True, False])
def test_key_weights_of_growing_and_falling_scores(dtype, D, up):
    """Key rows of growing (falling) length: the largest score of a row comes
    last (first), hundreds above the others."""
    import torch

    def edit(ck, Q, co):
        blk = _block(ck, co, 0, 2)
        n = blk.shape[1]
        f = torch.linspace(0.01, 6.0, n, device="cuda")
        blk.mul_((f if up else f.flip(0))[None, :, None].to(blk.dtype))

    _weights_case(1, 2, 4, D, dtype, prefix=[900], q=[3], spread=1.7, edit=edit)


def test_key_weights_flags_bad_input():
    from rag_precomputed_kv_gb300 import kvr
    for dtype, D in (("bf16", 128), ("fp32", 64)):
        def edit(ck, Q, co):
            Q[0, 0, 1, 3] = float("inf")
        with pytest.raises(kvr.KvrError) as e:
            _weights_case(1, 2, 2, D, dtype, prefix=[150], q=[2], edit=edit)
        assert e.value.status == 6


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def _evict_case(L, H, D, dtype, n, keep, first=0, recent=0, il=False, theta=THETA, in_place=False, keep_rotation=False,
                weights=None, spare=5, no_dst_weights=False, seed=1):
    import torch
    B, LH = len(n), L * H
    co = _starts([x + spare for x in n])
    k = [min(a, b) for a, b in zip(keep, n)]
    do = co if in_place else _starts([x + 2 for x in k])
    ck, cv = (_randn(seed + i, (int(co[-1]) * LH, D), dtype) for i in (0, 1))
    w = torch.exp(2 * _randn(seed + 2, (int(co[-1]) * LH,), "fp32"))
    if weights is not None:
        weights(w, co, LH)
    pool = _pool(L, H, 2, D, dtype, il, theta)
    kept = torch.full((max(1, sum(k) * LH),), -1, device="cuda", dtype=torch.int32)
    ck0, cv0, w0 = to_np64(ck), to_np64(cv), w.cpu().numpy()
    if in_place:
        dk, dv, dw = ck, cv, w
        got = pool.evict(co, n, keep, w, ck, cv, kept, n_first=first, n_recent=recent, keep_rotation=keep_rotation)
    else:
        dk, dv = (torch.full((int(do[-1]) * LH, D), float("nan"), device="cuda", dtype=_dt(dtype)) for _ in range(2))
        dw = None if no_dst_weights else torch.full((int(do[-1]) * LH,), float("nan"), device="cuda")
        got = pool.evict(co, n, keep, w, ck, cv, kept, dst_offsets=do, dst_k=dk, dst_v=dv, dst_weights=dw, n_first=first,
                         n_recent=recent, keep_rotation=keep_rotation)
    assert got.tolist() == k
    torch.cuda.synchronize()
    pool.check()
    kept = kept.cpu().numpy()
    at = 0
    for b in range(B):
        for u in range(LH):
            row = lambda x: _block(x, co, b, LH)[u]
            ww = row(w0)[:n[b]].astype(np.float64)
            rank = np.where(np.isnan(ww), -np.inf, ww)
            nan = np.isnan(ww)
            i = np.arange(n[b])
            must = (i < first) | (i >= n[b] - recent)
            # most wanted first: protected, numbers before NaN, heavier, lower row
            order = np.lexsort((i, -rank, nan, ~must))
            want = np.sort(order[:k[b]])
            mine = kept[at:at + k[b]]
            at += k[b]
            assert np.array_equal(mine, want), (b, u)
            gk, gv = to_np64(_block(dk, do, b, LH)[u]), to_np64(_block(dv, do, b, LH)[u])
            K, V = row(ck0)[want], row(cv0)[want]
            assert np.array_equal(gv[:k[b]], V)
            ref = K if keep_rotation else oracle.rope(K, (np.arange(k[b]) - want).astype(np.float64), theta, il)
            if keep_rotation:
                assert np.array_equal(gk[:k[b]], ref)
            elif k[b]:
                assert k_within_tolerance(gk[:k[b]], ref, dtype, il)[0]
            if dw is not None:
                gw = _block(dw, do, b, LH)[u].cpu().numpy()
                assert np.array_equal(gw[:k[b]], row(w0)[want], equal_nan=True)
                assert (gw[k[b]:] == 0).all()
            if in_place:   # rows behind the kept ones are left as they were
                assert np.array_equal(gk[k[b]:], row(ck0)[k[b]:]) and np.array_equal(gv[k[b]:], row(cv0)[k[b]:])
            else:
                assert np.isnan(gk[k[b]:]).all() and np.isnan(gv[k[b]:]).all()


EVICT = {
    "one-row": dict(n=[1], keep=[1]),
    "to-one": dict(n=[77], keep=[1]),
    "to-none": dict(n=[77, 3], keep=[0, 2]),
    "nothing-to-do": dict(n=[40, 200], keep=[40, 1000]),
    "empty-request": dict(n=[0, 150], keep=[8, 64]),
    "half": dict(n=[257, 1000, 63], keep=[128, 500, 32], first=4, recent=16),
    "only-protected": dict(n=[300], keep=[48], first=32, recent=16),
    "all-but-one": dict(n=[129, 700], keep=[128, 699], first=3, recent=3),
    "long": dict(n=[9001], keep=[4500], first=4, recent=64),
    "many": dict(n=[30 + 3 * i for i in range(70)], keep=[25 + i for i in range(70)], first=2, recent=3),
}


@pytest.mark.parametrize("name", EVICT)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H,D,dtype", [(2, 128, "bf16"), (1, 64, "fp32")])
def test_evict(name, in_place, H, D, dtype):
    _evict_case(1, H, D, dtype, in_place=in_place, **EVICT[name])


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp32"), (128, "bf16")])
def test_evict_interleaved_pairs_and_kept_rotation(D, dtype):
    _evict_case(2, 2, D, dtype, [6000, 90], [300, 50], 1, 2, il=True, theta=1e4)
    _evict_case(1, 2, D, dtype, [600, 90], [300, 50], 1, 2, keep_rotation=True, no_dst_weights=True)


@pytest.mark.parametrize("kind", ["equal", "two-values", "infinities", "nan", "zeros", "tiny"])
def test_evict_ties_and_special_weights(kind):
    import torch

    def weights(w, co, LH):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        r = torch.rand(w.shape, generator=g, device="cuda")
        if kind == "equal":
            w.fill_(0.25)
        elif kind == "two-values":
            w.copy_((r > 0.4).float())
        elif kind == "infinities":
            w[r > 0.9] = float("inf")
            w[r < 0.6] = -float("inf")
        elif kind == "nan":
            w[r > 0.3] = float("nan")
            w[r < 0.1] = -float("inf")
        elif kind == "zeros":
            w.copy_(torch.where(r > 0.5, 0.0, -0.0))
            w[r > 0.95] = -1.0
        else:
            w.copy_(r * 1e-42)

    for in_place in (False, True):
        _evict_case(1, 2, 128, "bf16", [1500, 200], [700, 60], 5, 7, weights=weights, in_place=in_place)
        _evict_case(1, 2, 128, "bf16", [1500, 200], [170, 60], 5, 7, weights=weights, in_place=in_place)


def test_evict_more_rows_than_shared_memory_holds():
    _evict_case(1, 1, 64, "bf16", [50001], [20000], 4, 64)
    _evict_case(1, 1, 64, "bf16", [60000], [333], 4, 64, in_place=True)


@pytest.mark.parametrize("heavy", [True, False])
@pytest.mark.parametrize("L,H,B,n,threads", [(1, 2, 1, 20000, 1024), (4, 8, 20, 3100, 256), (1, 1, 1, 51000, 1024)])
def test_evict_weights_unlike_their_sample(heavy, L, H, B, n, threads):
    """A first count of an eighth of the rows says where the threshold lies;
    here just those rows are the heavy (light) ones, and it lies elsewhere."""
    import torch

    def weights(w, co, LH):
        n_r = -(-n // threads)
        i = torch.arange(n, device="cuda")
        counted = (i % (32 * n_r)) // 32 % 8 == 0
        for b in range(B):
            blk = _block(w, co, b, LH)[:, :n]
            blk.mul_(torch.where(counted == heavy, 1e6, 1e-6))

    _evict_case(L, H, 64, "bf16", [n] * B, [n // 2] * B, 3, 5, weights=weights)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp32")])
def test_prefill_weights_evict_decode(D, dtype):
    """A prefill, the weights its last tokens give the cached keys, the cache
    cut to a budget, two decode steps on what is left."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, E, B, lq, win, keep = 2, 2, 4, 96, 3, 20, 8, 64
    rng = np.random.default_rng(3)
    pk, pv = _randn(1, (4, L, H, E, D), dtype), _randn(2, (4, L, H, E, D), dtype)
    pool = kvr.Pool(pk, pv, H * G, THETA)
    spans, so = [], [0]
    for b in range(B):
        for _ in range(4 + b):
            s = int(rng.integers(0, 40))
            spans.append((int(rng.integers(0, 4)), s, s + int(rng.integers(10, 50))))
        so.append(len(spans))
    P = np.array([sum(e - s for _, s, e in spans[so[b]:so[b + 1]]) for b in range(B)])
    co, qo = _starts(P + lq), (np.arange(B + 1) * lq).astype(np.int32)
    LH, dt = L * H, _dt(dtype)
    ck, cv = (torch.zeros((int(co[-1]) * LH, D), device="cuda", dtype=dt) for _ in range(2))
    q, kq, vq = _randn(3, (L, B * lq, H * G, D), dtype), _randn(4, (L, B * lq, H, D), dtype), _randn(5, (L, B * lq, H, D), dtype)
    out = torch.empty_like(q)
    assert (pool.prefill(so, spans, co, ck, cv, qo, q, kq, vq, out) == P).all()
    # the last `win` query tokens of each request
    sel = torch.cat([torch.arange(b * lq + lq - win, (b + 1) * lq) for b in range(B)]).cuda()
    w = torch.zeros(int(co[-1]) * LH, device="cuda")
    pool.key_weights(co, P + lq - win, (np.arange(B + 1) * win).astype(np.int32), q[:, sel].contiguous(), ck, w)
    n = P + lq
    do = _starts([keep + 2] * B)
    dk, dv = (torch.zeros((int(do[-1]) * LH, D), device="cuda", dtype=dt) for _ in range(2))
    dw = torch.empty(int(do[-1]) * LH, device="cuda")
    kept = torch.empty(B * keep * LH, device="cuda", dtype=torch.int32)
    m = pool.evict(co, n, [keep] * B, w, ck, cv, kept, dst_offsets=do, dst_k=dk, dst_v=dv, dst_weights=dw, n_first=4, n_recent=win)
    assert m.tolist() == [keep] * B
    outs, steps = [], []
    for step in range(2):
        x = (_randn(10 + step, (L, B, H * G, D), dtype), _randn(20 + step, (L, B, H, D), dtype), _randn(30 + step, (L, B, H, D), dtype))
        o = torch.empty_like(x[0])
        pool.query_attention(do, m + step, np.arange(B + 1), *x, dk, dv, o)
        pool.key_weights(do, m + step, np.arange(B + 1), x[0], dk, dw, accumulate=True)
        outs.append(o)
        steps.append(x)
    torch.cuda.synchronize()
    pool.check()
    kept = kept.cpu().numpy().reshape(B, LH, keep)
    for b in range(B):
        K0, V0 = to_np64(_block(ck, co, b, LH)), to_np64(_block(cv, co, b, LH))
        wb = _block(w, co, b, LH).cpu().numpy()
        db = to_np64(_block(dw, do, b, LH))
        for u in range(LH):
            l, h = divmod(u, H)
            # the weights of a window sum to its number of query rows
            assert abs(wb[u, :n[b]].sum() - win * G) < 1e-3
            i = np.arange(n[b])
            must = (i < 4) | (i >= n[b] - win)
            want = np.sort(np.lexsort((i, -wb[u, :n[b]].astype(np.float64), ~must))[:keep])
            assert np.array_equal(kept[b, u], want)
            K = oracle.rope(K0[u, want], (np.arange(keep) - want).astype(np.float64), THETA)
            V = V0[u, want]
            for step, (x, o) in enumerate(zip(steps, outs)):
                kr = oracle.rope(to_np64(x[1][l, b, h])[None], float(keep + step), THETA)
                K, V = np.concatenate([K, kr]), np.concatenate([V, to_np64(x[2][l, b, h])[None]])
                qr = oracle.rope(to_np64(x[0][l, b, h * G:(h + 1) * G])[None], float(keep + step), THETA)
                ref, A, qk, p = _attention_ref(K, V, qr, 0, keep + step, D ** -0.5)
                # keys of the evicted cache are rounded too: d holds a query and a key rounding
                _check_attention(to_np64(o[l, b, h * G:(h + 1) * G])[None], ref, A, qk, len(K), dtype, D)
            assert abs(db[u].sum() - (wb[u, want].sum() + 2 * G)) < 1e-3


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp32")])
def test_shared_prefix_decodes_as_one_cache(D, dtype):
    """Groups stitched once, a query prefill and decode steps over the shared
    prefix, against kvr_query_attention on caches that hold prefix and own rows
    one behind the other; then the own rows are evicted and decoding goes on."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, E = 2, 2, 4, 160
    pk, pv = _randn(1, (3, L, H, E, D), dtype), _randn(2, (3, L, H, E, D), dtype)
    pool = kvr.Pool(pk, pv, H * G, THETA)
    spans = [(0, 0, 100), (2, 17, 160), (1, 5, 60), (0, 3, 90)]
    so, go = [0, 2, 4], [0, 2, 5]
    P = np.array([243, 142], np.int32)
    B, LH, dt = 5, L * H, _dt(dtype)
    grp = [0, 0, 1, 1, 1]
    lq = [30, 1, 12, 40, 5]
    po = _starts(P)
    zeros = lambda rows: torch.zeros((int(rows) * LH, D), device="cuda", dtype=dt)
    gk, gv = zeros(po[-1]), zeros(po[-1])
    assert (pool.assemble(so, spans, po, gk, gv) == P).all()
    co, fo = _starts([n + 4 for n in lq]), _starts([P[grp[b]] + lq[b] + 4 for b in range(B)])
    ck, cv, fk, fv = zeros(co[-1]), zeros(co[-1]), zeros(fo[-1]), zeros(fo[-1])
    fso, fsp = [0], []
    for b in range(B):
        fsp += spans[so[grp[b]]:so[grp[b] + 1]]
        fso.append(len(fsp))
    fP = pool.assemble(fso, fsp, fo, fk, fv)
    own = np.zeros(B, np.int32)

    def step(qlen, seed):
        qo = _starts(qlen).astype(np.int32)
        x = [_randn(seed + i, (L, int(qo[-1]), H * (G if i == 0 else 1), D), dtype) for i in range(3)]
        o1, o2 = torch.empty_like(x[0]), torch.empty_like(x[0])
        pool.shared_query_attention(go, po, P, gk, gv, co, own, qo, *x, ck, cv, o1)
        pool.query_attention(fo, fP + own, qo, *x, fk, fv, o2)
        torch.cuda.synchronize()
        pool.check()
        own[:] += np.asarray(qlen, np.int32)
        a, b = to_np64(o1), to_np64(o2)
        # two results, each within its own bound of the exact one
        rel = np.linalg.norm(a - b) / np.linalg.norm(b)
        assert rel <= 2 * (3 ** 0.5 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17), rel
        for b in range(B):
            n0, n1 = int(P[grp[b]]), int(own[b])
            assert torch.equal(_block(ck, co, b, LH)[:, :n1], _block(fk, fo, b, LH)[:, n0:n0 + n1])
            assert torch.equal(_block(cv, co, b, LH)[:, :n1], _block(fv, fo, b, LH)[:, n0:n0 + n1])

    step(lq, 100)
    step([1] * B, 200)
    step([1, 0, 1, 1, 0], 300)
    # evict the own rows of both caches alike: the same rows by index, the full cache's behind its prefix
    w = torch.rand(int(co[-1]) * LH, device="cuda")
    keep = [min(10, int(x)) for x in own]
    kept = torch.empty(sum(keep) * LH, device="cuda", dtype=torch.int32)
    before = [(_block(ck, co, b, LH).clone(), _block(cv, co, b, LH).clone()) for b in range(B)]
    m = pool.evict(co, own, keep, w, ck, cv, kept, n_recent=1)
    torch.cuda.synchronize()
    at = 0
    for b in range(B):
        kb = kept[at:at + keep[b] * LH].view(LH, keep[b])
        at += keep[b] * LH
        n0 = int(P[grp[b]])
        for u in range(LH):
            rows = kb[u].long()
            assert torch.equal(_block(cv, co, b, LH)[u, :keep[b]], before[b][1][u][rows])
            _block(fk, fo, b, LH)[u, n0:n0 + keep[b]] = _block(ck, co, b, LH)[u, :keep[b]]
            _block(fv, fo, b, LH)[u, n0:n0 + keep[b]] = _block(cv, co, b, LH)[u, :keep[b]]
    own[:] = m
    step([1] * B, 400)


# ---------------------------------------------------------------------------
# streams, capture
# ---------------------------------------------------------------------------
def test_evict_and_weights_on_another_stream_and_in_a_graph():
    import torch
    L, H, G, D, n = 1, 2, 4, 128, 500
    pool = _pool(L, H, G, D, "bf16")
    from rag_precomputed_kv_gb300 import kvr
    ck, cv = _randn(1, (n * H, D), "bf16"), _randn(2, (n * H, D), "bf16")
    q = _randn(3, (L, 1, H * G, D), "bf16")
    w, kept = torch.zeros(n * H, device="cuda"), torch.zeros(100 * H, device="cuda", dtype=torch.int32)
    dk, dv, dw = torch.zeros((100 * H, D), device="cuda", dtype=ck.dtype), torch.zeros((100 * H, D), device="cuda", dtype=ck.dtype), torch.zeros(100 * H, device="cuda")

    def call():
        pool.key_weights([0, n], [n - 1], [0, 1], q, ck, w)
        pool.evict([0, n], [n], [100], w, ck, cv, kept, dst_offsets=[0, 100], dst_k=dk, dst_v=dv, dst_weights=dw, n_recent=4)

    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with pytest.raises(kvr.KvrError):      # not bound yet: refused, the capture stays usable
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            torch.zeros(1, device="cuda")
            call()
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in (w, kept, dk, dv, dw)]
    with torch.cuda.graph(g, stream=s):
        call()
    for x in (w, kept, dk, dv, dw):
        x.zero_()
    ck.copy_(ck.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(w, want[0])     # other inputs, other results
    ck.copy_(ck.flip(0))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip((w, kept, dk, dv, dw), want):
        assert torch.equal(x, y)
    for x in (w, kept, dk, dv, dw):
        x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    for x, y in zip((w, kept, dk, dv, dw), want):
        assert torch.equal(x, y)
    pool.check()


@pytest.mark.parametrize("D,dtype", [(64, "fp32"), (128, "bf16")])
def test_shared_prefix_in_a_graph(D, dtype):
    """The CUDA-core path is kernels alone and can be captured; the tensor-core
    path uses the pool's scratch and says so, and the capture stays usable."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    pool, args, _ = _shared_case(1, 2, 2, D, dtype, groups=[2], prefix=[140], own=[3, 0], q=[1, 1])
    want = args[-1].clone()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    if dtype == "bf16":
        with torch.cuda.graph(g, stream=s):
            args[-1].zero_()
            with pytest.raises(kvr.KvrError) as e:
                pool.shared_query_attention(*args)
        assert e.value.status == 3
        pool.shared_query_attention(*args)
    else:
        with torch.cuda.graph(g, stream=s):
            pool.shared_query_attention(*args)
        args[-1].zero_()
        g.replay()
    torch.cuda.synchronize()
    pool.check()
    assert torch.equal(args[-1], want)


def test_caches_beyond_32_bit_offsets():
    """Blocks that begin 2^31 elements into their tensors give what they give at the start."""
    import torch
    L, H, G, D, far, n = 1, 1, 4, 128, (1 << 24) + 77, 400
    pool = _pool(L, H, G, D, "bf16")
    near = [_randn(i, (n, D), "bf16") for i in (1, 2)]
    big = [torch.empty((far + n, D), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    pk, pv = _randn(3, (200, D), "bf16"), _randn(4, (200, D), "bf16")
    q, kq, vq = _randn(5, (L, 1, G, D), "bf16"), _randn(6, (L, 1, H, D), "bf16"), _randn(7, (L, 1, H, D), "bf16")
    got = []
    for ck, cv, o in ((*[x.clone() for x in near], 0), (*big, far)):
        if o:
            ck[o:], cv[o:] = near[0], near[1]
        w = torch.zeros(o + n, device="cuda")
        kept = torch.empty(100, device="cuda", dtype=torch.int32)
        out = torch.empty_like(q)
        co = [o, o + n]
        pool.shared_query_attention([0, 1], [0, 200], [200], pk, pv, co, [n - 10], [0, 1], q, kq, vq, ck, cv, out)
        pool.key_weights(co, [n - 10], [0, 1], q, ck, w)
        pool.evict(co, [n - 9], [100], w, ck, cv, kept, n_first=3, n_recent=5)
        torch.cuda.synchronize()
        pool.check()
        got.append([x.clone() for x in (out, w[o:], kept, ck[o:], cv[o:])])
    for x, y in zip(*got):
        assert torch.equal(x, y)
