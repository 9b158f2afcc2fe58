"""How near the paged attention's kernels come to fp64, each by its own precision, and
queries and scales at the ends of fp32's range.

A result rounded to bf16 is off by r = ||round(o) - o|| / ||o||, which is taken from the
fp64 result itself.  Each operand that a kernel rounds to bf16 on the way (the turned
query, the probability, a restored key, a restored value) is off by as much in the rms
and independently of the others: with queries and keys of unit variance a score's error
is r times its own spread of 1, and so is the probability's.  n roundings give r sqrt(n):
    up to 16 query rows, bf16 rows             n = 1   the output alone
    up to 16, or in parts, on packed rows      n = 2   and the probability times its scale
    more query rows                            n = 3   the output, the query, the probability
    more query rows on packed rows             n = 5   and keys and values, restored
(fp16 queries, 11 bits, add 1/64.)  The limit is half a rounding above, r sqrt(n + 1/2):
one rounding more does not pass.
"""
import numpy as np
import pytest

from test_gpu_page_cache import THETA, _packed_ref, _pool, _randn, _starts, _table

pytestmark = pytest.mark.gpu


def _turn64(x, pos, theta=THETA):
    """x [..., T, heads, D] fp64 on the GPU, token t turned by pos[t]."""
    import torch
    h = x.shape[-1] // 2
    w = theta ** (-torch.arange(h, dtype=torch.float64, device=x.device) / h)
    a = torch.as_tensor(np.asarray(pos), dtype=torch.float64, device=x.device)[:, None, None] * w
    lo, hi = x[..., :h], x[..., h:]
    return torch.cat([lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()], -1)


def _rows64(x, ids, n, R):
    """Rows 0 .. n - 1 through the pages `ids`: [L, H, n, D] in fp64."""
    import torch
    return torch.cat([x[int(i)] for i in ids[:-(-n // R)]], 2)[:, :, :n].double()


def _thin64(x):
    """What the packed form of bf16 rows stands for, exactly."""
    code, scale = _packed_ref(x.to("cpu"))
    return (code * scale).reshape(x.shape).to("cuda")


def _attend64(q, K, V, pos, scale):
    """q [L, T, Hq, D] turned, K, V [L, H, n, D]; every token sees rows <= its position."""
    import torch
    L, T, Hq, D = q.shape
    H, n = K.shape[1], K.shape[2]
    x = q.view(L, T, H, Hq // H, D)
    hide = torch.arange(n, device="cuda") > torch.as_tensor(np.asarray(pos), device="cuda")[:, None]
    out = torch.empty_like(x)
    for l in range(L):
        for h in range(H):
            s = torch.einsum("tgd,nd->tgn", x[l, :, h], K[l, h]) * scale
            s.masked_fill_(hide[:, None], -float("inf"))
            out[l, :, h] = torch.einsum("tgn,nd->tgd", torch.softmax(s, -1), V[l, h])
    return out.view(L, T, Hq, D)


def _off(got, want):
    """||got - want|| / ||want|| and the same of want rounded to bf16."""
    import torch
    n = want.norm()
    return float((got.double() - want).norm() / n), float((want.to(torch.bfloat16).double() - want).norm() / n)


def _case(reqs, G, L=2, H=4, R=64, seed=1):
    """reqs: (rows, query tokens, packed rows, roundings).  Each request against its own limit."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    D = 128
    kv, lq, body, roundings = (list(x) for x in zip(*reqs))
    t, n = _table(kv, R, seed)
    k, v = (_randn(seed + i, (n, L, H, R, D), "bf16") for i in (1, 2))
    Q = _randn(seed + 3, (L, sum(lq), H * G, D), "bf16")
    out = torch.full_like(Q, float("nan"))
    pool, kw = _pool(L, H, G, D, "bf16"), {}
    if any(body):
        packed = pool.packed_pages(n, R)
        pool.page_pack(kvr.Pages(k, v), t, packed, t, [0] * len(body), body)
        kw = dict(packed=packed, packed_table=t, packed_len=body)
    qo = _starts(lq)
    pool.page_attention(kvr.Pages(k, v), t, kv, qo.astype(np.int32), Q, out, **kw)
    pool.check()
    for b, (m, T, p, roundings) in enumerate(reqs):
        a, e = int(qo[b]), int(qo[b + 1])
        pos = m - T + np.arange(T)
        K, V = _rows64(k, t[b], m, R), _rows64(v, t[b], m, R)
        if p:
            K[:, :, :p], V[:, :, :p] = (_thin64(_rows64(x, t[b], p, R).to(torch.bfloat16)) for x in (k, v))
        want = _attend64(_turn64(Q[:, a:e].double(), pos), K, V, pos, D ** -0.5)
        off, r = _off(out[:, a:e], want)
        assert 0.8 * r <= off <= r * np.sqrt(roundings + 0.5), (b, off, r, off * off / (r * r))
    return pool


@pytest.mark.parametrize("G,q", [(1, 16), (4, 1), (4, 4), (7, 2), (8, 1), (16, 1)])
def test_few_query_rows_are_off_by_their_rounding(G, q):
    _case([(700, q, 0, 1), (333, q, 0, 1), (1500, 1, 0, 1)], G)


@pytest.mark.parametrize("G,q", [(1, 16), (4, 1), (4, 4), (7, 2), (16, 1), (1, 17), (1, 48), (4, 12), (7, 6), (16, 3)])
def test_few_query_rows_and_parts_on_packed_rows(G, q):
    """... in parts as alone, and one that sees no packed row beside them as without them."""
    _case([(700, q, 640, 2), (333, q, 320, 2), (900, 1, 0, 1), (1500, 1, 1472, 2)], G)


@pytest.mark.parametrize("G,q", [(1, 17), (4, 40), (7, 64), (16, 2), (20, 1)])
def test_many_query_rows(G, q):
    _case([(700, q, 0, 3), (333, q, 0, 3), (1500, q, 0, 3)], G)


@pytest.mark.parametrize("G,q", [(1, 49), (4, 13), (7, 64), (16, 4), (20, 1)])
def test_many_query_rows_on_packed_rows(G, q):
    _case([(700, q, 640, 5), (333, q, 320, 5), (1500, q, 1408, 5)], G)


def test_each_request_of_a_call_keeps_its_own_precision():
    _case([(700, 60, 640, 5), (700, 60, 0, 3), (700, 1, 640, 2), (700, 12, 640, 2), (700, 1, 0, 1)], 4)


# ---------------------------------------------------------------------------
# the ends of fp32's range
# ---------------------------------------------------------------------------
def _end_case(G, q, scale, make, body, R=32, n=200, window=0, first=0):
    """Queries [T, heads, D] and rows [n, D] by make(pos): output, values seen by each token."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    D = 128
    t, pages = _table([n], R, 3)
    pos = n - q + np.arange(q)
    Q, K = make(pos)
    k = torch.zeros((pages, 1, 1, R, D), device="cuda", dtype=torch.bfloat16)
    v = _randn(5, (pages, 1, 1, R, D), "bf16")
    for r in range(n):
        k[int(t[0, r // R]), 0, 0, r % R] = K[r]
    pool = _pool(1, 1, G, D, "bf16")
    kw = {}
    if body:
        packed = pool.packed_pages(pages, R)
        pool.page_pack(kvr.Pages(k, v), t, packed, t, [0], [body])
        kw = dict(packed=packed, packed_table=t, packed_len=[body])
    out = torch.full((1, q, G, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    pool.page_attention(kvr.Pages(k, v), t, [n], [0, q], Q[None].contiguous(), out, softmax_scale=scale, window=window, n_first=first, **kw)
    pool.check()
    V = _rows64(v, t[0], n, R)
    if body:
        V[:, :, :body] = _thin64(V[:, :, :body].to(torch.bfloat16))
    return out[0].double(), V[0, 0], pos


@pytest.mark.parametrize("q,G", [(1, 1), (3, 4), (9, 4), (20, 4)])
@pytest.mark.parametrize("scale", [0.0, 1e-7, 1e-8, 1e-20, 1e-40])
@pytest.mark.parametrize("body", [0, 160])
def test_queries_of_zeros_weigh_all_rows_alike(q, G, scale, body):
    """... whatever the scale, in tiles with hidden rows too: the mean of the values that are seen."""
    import torch
    zeros = lambda pos: (torch.zeros((q, G, 128), device="cuda", dtype=torch.bfloat16), _randn(7, (200, 128), "bf16"))
    for window, first in ((0, 0), (77, 5)):
        got, V, pos = _end_case(G, q, scale, zeros, body, window=window, first=first)
        for i, p in enumerate(pos):
            rows = np.arange(200)
            seen = (rows <= p) & ((rows > p - window) | (rows < first)) if window else rows <= p
            W = V[torch.from_numpy(seen).cuda()]
            # probabilities of 1 (or, on packed rows, a scale) are exact: the output's rounding, and sums in fp32;
            # restored values are rounded once more
            bound = 2.0 ** -8 * W.mean(0).abs() + W.abs().mean(0) * (2.0 ** -8 * bool(body) + 200 * 2.0 ** -22)
            assert ((got[i] - W.mean(0)).abs() <= bound).all()


@pytest.mark.parametrize("top,body", [(-113, 160), (-100, 0), (-100, 160), (-60, 160), (60, 160), (100, 160), (100, 0), (119, 0), (122, 0)])
def test_large_and_small_queries_meet_keys_that_undo_them(top, body):
    """Queries of 2^top in one pair of dims, keys of 0, 1 or 2 times +-2^-top there, whose scores are ordinary."""
    import torch
    q, G, n = 3, 4, 200

    def make(pos):
        Q = torch.zeros((q, G, 128), device="cuda", dtype=torch.float64)
        Q[..., 0] = 2.0 ** top
        # (keys in the direction of the middle token, whose angle the others miss by a radian)
        w = ((torch.arange(n, device="cuda") * 7919) % 5 - 2).double() * 2.0 ** -top
        K = torch.zeros((n, 128), device="cuda", dtype=torch.float64)
        K[:, 0], K[:, 64] = w * np.cos(pos[1]), w * np.sin(pos[1])
        make.K = K.to(torch.bfloat16)
        return Q.to(torch.bfloat16), make.K

    got, V, pos = _end_case(G, q, 1.0, make, body, n=n)
    K = make.K.double()
    if body:
        K[:body] = _thin64(make.K[:body])
    for i, p in enumerate(pos):
        d = torch.zeros(128, device="cuda", dtype=torch.float64)
        d[0], d[64] = np.cos(p) * 2.0 ** top, np.sin(p) * 2.0 ** top
        w = torch.softmax(K[:p + 1] @ d, 0)
        want, A = w @ V[:p + 1], w @ V[:p + 1].abs()
        # the output's rounding; scores of at most 2, off by the query's 2^-11, move a weight by twice that; the
        # rounding of probabilities on packed rows; sums
        bound = 2.0 ** -8 * want.abs() + A * (2.0 ** -8 * bool(body) + 2.1 * 2 * 2.0 ** -11 + 200 * 2.0 ** -22)
        assert ((got[i] - want).abs() <= bound).all()


@pytest.mark.parametrize("top", [100, 119, 122])
@pytest.mark.parametrize("body", [0, 160])
def test_a_score_far_above_the_others_takes_all(top, body):
    """Queries of 2^top against keys of -1, 1 and, once, 2 in the same pair: the value of that row, or a report."""
    import torch
    q, G, n, best = 2, 4, 200, 33

    def make(pos):
        Q = torch.zeros((q, G, 128), device="cuda", dtype=torch.float64)
        Q[..., 0] = 2.0 ** top
        c = (torch.arange(n, device="cuda") % 2 * 2 - 1).double()
        c[best] = 2.0
        K = torch.zeros((n, 128), device="cuda", dtype=torch.float64)
        K[:, 0], K[:, 64] = c * np.cos(pos[0]), c * np.sin(pos[0])   # (half as much for the second token, a radian off)
        return Q.to(torch.bfloat16), K.to(torch.bfloat16)

    # the step of a score beyond 2^30 in fp32 is above 2^6: a weight of such a maximum may pass fp32's range,
    # which is reported
    from rag_precomputed_kv_gb300 import kvr
    try:
        got, V, _ = _end_case(G, q, 1.0, make, body, n=n)
    except kvr.KvrError as e:
        assert e.status == 6
    else:
        assert ((got - V[best]).abs() <= 2.0 ** -8 * V[best].abs() + 2.0 ** -22).all()


@pytest.mark.parametrize("top", [117, 122])
def test_queries_beyond_the_range_on_packed_rows_are_reported(top):
    import torch
    from rag_precomputed_kv_gb300 import kvr

    def make(pos):
        Q = torch.full((2, 4, 128), 2.0 ** top, device="cuda", dtype=torch.bfloat16)
        return Q, _randn(7, (200, 128), "bf16", 2.0 ** -top)

    with pytest.raises(kvr.KvrError) as e:
        _end_case(4, 2, 1.0, make, 160)
    assert e.value.status == 6
