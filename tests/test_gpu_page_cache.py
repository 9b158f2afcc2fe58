"""The paged cache on the GPU against plain fp64 numpy (rotations of the oracle).

Tolerances, in half steps u of a type (bf16 2^-8, fp32 2^-24) relative to a
value:
* appended keys: the stitched keys' tolerance; values and all other rows: exact.
* packed rows: their codes and scales are whole multiples and bf16 numbers that
  any correct rounding gives, so restored rows are exactly scale * code rounded
  to bf16.
* attention, with A = sum_j p_j |v_j| and d the largest change that rounding can
  make to a score of the row,
      |o - o_ref| <= u |o_ref| + A ((1 + u)^r e^{2d} - 1) + n 2^-22 A:
  one rounding of the output, r of each weighted value, a score off by d moves p
  by at most e^{+-2d}, and sums of n terms in fp32.  With e the rounding of the
  query, d = scale sum_i |q_i k_i| (e + (D + 8) 2^-24) (D products and a rotation of
  4 roundings each way in fp32):
      fp32, and bf16 with head_dim 64              e = 0        r = 0
      bf16, up to 16 rows a request                e = 2^-11    r = 2^-8 (16 bits)
        that see packed rows (up to three parts)   e = 2^-11    r = 1
      more rows                                    e = u        r = 1
        that see packed rows (rounded to bf16)     e = 2 u      r = 2
  In the 2-norm the roundings are independent and add in squares: of the output,
  the query or key, the probability, the value, each u: ||o - o_ref|| <= sqrt(k) u ||o_ref||,
  k = 1.1, 1.1, 2.2, 3 and 5 in bf16 (1.1, 2.2: with what the others leave); in fp32
  2^-17 ||o_ref|| (scores off by up to 2^-17).
"""
import gc

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


def _table(rows, R, seed=0, spare=2):
    """Pages for requests of so many rows, shuffled; -1 behind them."""
    need = [-(-r // R) for r in rows]
    ids = np.random.default_rng(seed).permutation(sum(need) + spare).astype(np.int32)
    t = np.full((len(rows), max(need + [1])), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, sum(need) + spare


def _rows(x, t, b, rows, R):
    """Rows of request b of pages x [n, L, H, R, D] (numpy): [L, H, rows, D]."""
    rows = np.asarray(rows, np.int64)
    return np.moveaxis(x[t[b, rows // R], :, :, rows % R], 0, 2)


def _turned(x, pos, il, theta=THETA):
    """x [L, T, heads, D] turned token by token."""
    return oracle.rope(x, np.asarray(pos, np.float64)[None, :, None], theta, interleaved=il)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _append_case(dtype, D, R, start, q, L=2, H=2, G=2, il=False, turned=False, strided=False, seed=1, stream=None, pool=None):
    import torch
    from rag_precomputed_kv_gb300 import kvr
    T = sum(q)
    t, n = _table([a + b for a, b in zip(start, q)], R, seed)
    k, v = (_randn(seed + i, (n, L, H, R, D), dtype) for i in (0, 1))
    k[0], v[-1] = float("nan"), float("inf")         # rows nobody appends to stay, whatever they hold
    nk, nv = (_randn(seed + i, (L, H, T, D), dtype).transpose(1, 2) if strided else _randn(seed + i, (L, T, H, D), dtype) for i in (2, 3))
    k0, v0 = k.clone(), v.clone()
    torch.cuda.synchronize()
    pool = pool or _pool(L, H, G, D, dtype, il)
    pool.page_append(kvr.Pages(k, v), t, start, _starts(q).astype(np.int32), nk, nv, turned=turned, stream=stream)
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(a, a + b) for a, b in zip(start, q)] + [np.zeros(0, np.int64)]).astype(np.int64)
    page = np.concatenate([t[b, np.arange(a, a + n_) // R] for b, (a, n_) in enumerate(zip(start, q))] + [np.zeros(0, np.int64)]).astype(np.int64)
    mine = np.zeros((n, R), bool)
    mine[page, pos % R] = True
    keep = torch.from_numpy(~mine).cuda()
    for x, x0 in ((k, k0), (v, v0)):
        a, b = (y.permute(0, 3, 1, 2, 4)[keep].contiguous().view(torch.int16 if dtype == "bf16" else torch.int32) for y in (x, x0))
        assert torch.equal(a, b)
    if T == 0:
        return
    got_k, got_v = (y.permute(0, 3, 1, 2, 4)[torch.from_numpy(page).cuda(), torch.from_numpy(pos % R).cuda()] for y in (k, v))   # [T, L, H, D]
    assert torch.equal(got_v, nv.transpose(0, 1))
    if turned:
        assert torch.equal(got_k, nk.transpose(0, 1))
    else:
        ref = _turned(to_np64(nk), pos, il)
        got = to_np64(got_k).transpose(1, 0, 2, 3)
        ok, worst = k_within_tolerance(got, ref, dtype, il)
        assert ok, worst


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("il", [False, True])
def test_append_types_and_layouts(dtype, D, il):
    _append_case(dtype, D, 16, [0, 7, 4095, 100], [1, 30, 3, 0], il=il)
    _append_case(dtype, D, 64, [65, 0], [1, 200], L=3, H=1, G=5, il=il, strided=True, seed=3)


@pytest.mark.parametrize("R", [1, 3, 20, 48, 256])
def test_append_page_sizes(R):
    _append_case("bf16", 128, R, [0, R - 1, 5 * R], [2 * R + 1, 2, 1])
    _append_case("bf16", 128, R, [0, 11], [150, 40], turned=True, strided=True, seed=5)


def test_append_many_requests_and_far_positions():
    _append_case("bf16", 128, 32, [(i * 37) % 300 for i in range(150)], [i % 3 for i in range(150)])      # uploaded tables
    _append_case("bf16", 128, 1 << 20, [(1 << 24) - 5, 8191], [5, 1], L=1, H=1)
    _append_case("bf16", 128, 16, [20000], [3], L=1)                                                         # 1,251 pages of table


def test_append_nothing():
    _append_case("bf16", 128, 16, [3, 9], [0, 0])


def test_append_into_pages_of_other_strides():
    """Key and value pages side by side in one tensor; a flat block as pages."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, R, D, n = 2, 3, 16, 128, 5
    pool = _pool(L, H, 2, D, "bf16")
    both = _randn(1, (n, 2, L, H, R, D), "bf16")
    nk, nv = _randn(2, (L, 20, H, D), "bf16"), _randn(3, (L, 20, H, D), "bf16")
    pool.page_append(kvr.Pages(both[:, 0], both[:, 1]), [[3, 1]], [7], [0, 20], nk, nv, turned=True)
    flat_k, flat_v = _randn(4, (L, H, n * R, D), "bf16"), _randn(5, (L, H, n * R, D), "bf16")
    k0 = flat_k.clone()
    pages = kvr.Pages(*(x.view(L, H, n, R, D).permute(2, 0, 1, 3, 4) for x in (flat_k, flat_v)))
    pool.page_append(pages, [list(range(n))], [7], [0, 20], nk, nv, turned=True)
    torch.cuda.synchronize()
    assert torch.equal(both[3, 0, :, :, 7:], nk[:, :9].transpose(1, 2)) and torch.equal(both[1, 1, :, :, :11], nv[:, 9:].transpose(1, 2))
    assert torch.equal(flat_k[:, :, 7:27], nk.transpose(1, 2)) and torch.equal(flat_v[:, :, 7:27], nv.transpose(1, 2))
    assert torch.equal(flat_k[:, :, :7], k0[:, :, :7]) and torch.equal(flat_k[:, :, 27:], k0[:, :, 27:])


# ---------------------------------------------------------------------------
# pack and unpack
# ---------------------------------------------------------------------------
def _bf16(x):
    """fp64 to the nearest bf16, halves to even (a value an exact multiple of its step / 2^16)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).float().to(torch.bfloat16)


def _packed_ref(x):
    """(codes, scales) of bf16 rows x [..., 128] (torch, CPU), by the definition in 64 bits."""
    import torch
    y = x.double().reshape(*x.shape[:-1], 4, 32)
    top = y.abs().amax(-1, keepdim=True)
    fin = torch.isfinite(y).all(-1, keepdim=True)
    scale = torch.where(fin, (torch.where(fin, top, 0.0).float() / 7.0).to(torch.bfloat16).double(), float("nan"))
    code = torch.where(scale > 0, torch.round(y / torch.where(scale > 0, scale, 1.0)), 0.0).clamp(-7, 7)
    return code, scale


def _pack_case(R, begin, end, L=2, H=2, seed=1, data=None, stride_from=None):
    import torch
    from rag_precomputed_kv_gb300 import kvr
    D = 128
    t, n = _table([e + 5 for e in end], R, seed)
    tp, npk = _table(end, R, seed + 1)
    k, v = (_randn(seed + i, (n, L, H, R, D), "bf16") for i in (2, 3))
    if data is not None:
        k, v = data(k), data(v)
    pool = _pool(L, H, 2, D, "bf16")
    pages, packed = kvr.Pages(k, v), pool.packed_pages(npk, R)
    packed.data.fill_(0x5a)
    pool.page_pack(pages, t, packed, tp, begin, end)
    torch.cuda.synchronize()
    # only the blocks of these rows were written
    blocks = packed.data.view(npk, L, H, R // 32, 4608).cpu()
    mine = np.zeros((npk, R // 32), bool)
    for b in range(len(end)):
        for r in range(begin[b], end[b], 32):
            mine[tp[b, r // R], r % R // 32] = True
    assert (blocks.permute(0, 3, 1, 2, 4)[torch.from_numpy(~mine)] == 0x5a).all()
    k2, v2 = (torch.full_like(x, 3.0) for x in (k, v))
    pool.page_unpack(packed, tp, kvr.Pages(k2, v2), t, begin, end)
    torch.cuda.synchronize()
    kc, vc, k2c, v2c = (x.cpu() for x in (k, v, k2, v2))
    for x, y in ((kc, k2c), (vc, v2c)):
        left = torch.ones((n, R), dtype=torch.bool)
        for b in range(len(end)):
            rows = np.arange(begin[b], end[b])
            if not len(rows):
                continue
            pg, r = torch.from_numpy(t[b, rows // R].astype(np.int64)), torch.from_numpy(rows % R)
            left[pg, r] = False
            code, scale = _packed_ref(x[pg, :, :, r])
            want = (code * scale).reshape(*code.shape[:-2], 128).float().to(torch.bfloat16)   # (11 bits: exact in fp32)
            got = y[pg, :, :, r]
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
        assert (y.permute(0, 3, 1, 2, 4)[left] == 3.0).all()


@pytest.mark.parametrize("R", [32, 64, 96, 256])
def test_pack_and_unpack(R):
    _pack_case(R, [0, 32, 0, 64], [64, 160, 0, 64 + 2 * 96])
    _pack_case(R, [0], [32], L=1, H=1, seed=7)


def test_pack_values_between_codes():
    """Exact halves, ties and values next to them: every 8-bit number over every scale."""
    import torch

    def data(x):
        y = x.reshape(-1, 32).clone()
        i = torch.arange(y.shape[0], device="cuda")
        top = (1.0 + (i % 128) / 128.0) * 2.0 ** ((i // 128) % 9 - 4).float()
        y[:, 0] = top.to(torch.bfloat16)
        scale = (y[:, 0].float() / 7).to(torch.bfloat16).float()
        for m in range(7):
            half = (scale * (m + 0.5)).to(torch.bfloat16)
            bits = half.view(torch.int16)
            for d in (-1, 0, 1):
                y[:, 1 + 3 * m + d + 1] = (bits + d).view(torch.bfloat16) * (1 if m % 2 else -1)
        return y.reshape(x.shape)

    _pack_case(64, [0, 0], [1024, 512], data=data)


def test_pack_special_values():
    import torch

    def data(x):
        y = x.clone()
        y[..., 0, 0] = float("nan")
        y[..., 1, 40] = float("inf")
        y[..., 2, 70] = -float("inf")
        y[..., 3, :] = 0.0
        y[..., 4, 96:] = -0.0
        y[..., 5, :] = 3.3895e38                       # the largest
        y[..., 6, :32] = 1.2e-38                       # scales below the normal numbers
        y[..., 7, :] *= 1e-39
        y[..., 8, :] = 9.2e-41                         # the smallest: its scale is 0
        y[..., 9, :] = 4.6e-40
        y[..., 10, 32:64] *= 1e-36
        return y

    _pack_case(32, [0, 32], [64, 96], data=data)


def test_pack_many_requests():
    _pack_case(32, [0] * 130, [32 * (i % 3) for i in range(130)], L=1, H=1)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attention_ref(K, V, q, rows, pos, hi, window, first, scale):
    """K, V [n, D] fp64 of `rows`; q [Lq, G, D] turned.  Outputs, A, sum |q k| (max over keys), rows that see something."""
    Lq, G = q.shape[:2]
    see = (rows[None, :] <= pos[:, None]) & (rows[None, :] < hi)
    if window:
        see &= (rows[None, :] > pos[:, None] - window) | (rows[None, :] < first)
    some = see.any(1)
    if not len(rows):
        z = np.zeros((Lq, G, q.shape[2]))
        return z, z, np.zeros((Lq, G)), some
    s = np.where(see[:, None], np.einsum("tgd,nd->tgn", q, K) * scale, -np.inf)
    p = np.exp(s - np.where(some[:, None, None], s.max(-1, keepdims=True), 0.0))
    p = p / np.where(some[:, None, None], p.sum(-1, keepdims=True), 1.0)
    qk = np.where(see[:, None], np.einsum("tgd,nd->tgn", np.abs(q), np.abs(K)), 0.0).max(-1) * scale
    return np.einsum("tgn,nd->tgd", p, V), np.einsum("tgn,nd->tgd", p, np.abs(V)), qk, some


def _attention_case(reqs, L=2, H=2, G=4, D=128, dtype="bf16", R=16, window=0, first=0, il=False, scale=0.0, spread=1.0, seed=1,
                    stream=None, pool=None, default_pos=False, in_place=False, theta=THETA, poison=True, twice=False, pad=0, parts=1):
    """reqs: (kv_len, first query's position, query tokens, packed rows) of each request."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    kv, pos, lq, body = (list(x) for x in zip(*reqs))
    hi = [min(k, p + n) for k, p, n in zip(kv, pos, lq)]
    lo = [min(h, max(0, p - window + 1)) if window else 0 for h, p in zip(hi, pos)]
    few = [min(first, x) for x in lo]
    seen = [np.r_[0:f, a:h] if n else np.r_[0:0] for f, a, h, n in zip(few, lo, hi, lq)]
    t, n = _table([max(k, 1) for k in kv], R, seed)
    k, v = (_randn(seed + i, (n, L, H, R, D), dtype, spread) for i in (2, 3))
    if pad:          # pages, layers and heads at odd distances
        strides = ((L * H * (R * D + pad) + pad) + pad, H * (R * D + pad) + pad, R * D + pad, D, 1)
        for x in (k, v):
            y = torch.empty(n * strides[0] + L * strides[1], device="cuda", dtype=x.dtype).as_strided(x.shape, strides)
            y.copy_(x)
            x.set_(y)
    pool = pool or _pool(L, H, G, D, dtype, il, theta)
    kw = {}
    held = [to_np64(x) for x in (k, v)]
    if any(body):
        tp, npk = _table([max(b, 1) for b in body], R, seed + 1)
        packed = pool.packed_pages(npk, R)
        packed.data.fill_(0xff)                                    # scales of NaN
        pool.page_pack(kvr.Pages(k, v), t, packed, tp, [0] * len(body), body)
        u = torch.empty_like(k), torch.empty_like(v)
        for x, y in zip((k, v), u):
            code, s = _packed_ref(x.cpu())
            y.copy_((code * s).reshape(x.shape).float())          # rounded: the exact values follow
        exact = [(_packed_ref(x.cpu())[0] * _packed_ref(x.cpu())[1]).reshape(x.shape).numpy() for x in (k, v)]
        kw = dict(packed=packed, packed_table=tp, packed_len=body)
        if poison:   # packed rows outside what is seen: scales of NaN again
            # [pages, L, H, 16 rows, keys or values, rows n and n + 8 by turns, groups]
            scales = packed.data.view(npk, L, H, R // 16, 2, 1152)[..., 1024:].view(torch.bfloat16).unflatten(-1, (8, 2, 4))
            for b in range(len(reqs)):
                gone = np.setdiff1d(np.arange(body[b]), seen[b])
                for r in gone:
                    scales[int(tp[b, r // R]), :, :, r % R // 16, :, r % 8, r % 16 // 8] = float("nan")
    T, qo = sum(lq), _starts(lq).astype(np.int32)
    if poison:       # nothing may come of rows that no query sees, nor of pages without one
        mask = torch.ones((n, R), dtype=torch.bool)
        for b in range(len(reqs)):
            rows = seen[b][seen[b] >= body[b]]
            mask[torch.from_numpy(t[b, rows // R].astype(np.int64)), torch.from_numpy(rows % R)] = False
        mask = mask.cuda()[:, None, None, :, None]
        k.masked_fill_(mask, float("nan"))
        v.masked_fill_(mask, float("inf"))
        for b in range(len(reqs)):
            for x, rows in ((t, seen[b][seen[b] >= body[b]]),) + (((tp, seen[b][seen[b] < body[b]]),) if any(body) else ()):
                drop = np.setdiff1d(np.arange(x.shape[1]), rows // R)
                x[b, drop] = -7
    Q = _randn(seed + 4, (L, T, H * G, D), dtype, spread)
    out = Q if in_place else torch.full_like(Q, float("nan"))
    qd = to_np64(Q)
    torch.cuda.synchronize()
    args = (kvr.Pages(k, v), t, kv, qo, Q, out)
    if not default_pos:
        kw["q_pos"] = pos
    for _ in range(2 if twice else 1):
        pool.page_attention(*args, window=window, n_first=first, softmax_scale=scale, stream=stream, **kw)
    torch.cuda.synchronize()
    pool.check()
    got = to_np64(out).reshape(L, T, H, G, D)
    sc = scale if scale > 0 else D ** -0.5
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    e2 = n2 = worst = 0.0
    t0, _ = _table([max(x, 1) for x in kv], R, seed)
    for b in range(len(reqs)):
        if not lq[b]:
            continue
        a, e = int(qo[b]), int(qo[b + 1])
        at = pos[b] + np.arange(lq[b])
        q = _turned(qd[:, a:e], at, il, theta).reshape(L, lq[b], H, G, D)
        thin = bool((seen[b] < body[b]).any())
        if dtype == "fp32" or D == 64:
            e_q, r, k = 0.0, 0.0, 1.1
        elif lq[b] * G <= 16 or parts > 1 and thin and -(-lq[b] // (16 // G)) <= parts:
            e_q, r, k = 2.0 ** -11, (1.0 if thin else u), (2.2 if thin else 1.1)
        else:
            e_q, r, k = u * (1 + thin), 1.0 + thin, (5.0 if thin else 3.0)
        worst = max(worst, k)
        for l in range(L):
            for h in range(H):
                K, V = (_rows(x[:, l:l + 1, h:h + 1], t0, b, seen[b], R)[0, 0] for x in held)
                if body[b]:
                    m = seen[b] < body[b]
                    for x, y in zip((K, V), exact):
                        x[m] = _rows(y[:, l:l + 1, h:h + 1], t0, b, seen[b][m], R)[0, 0]
                o, A, qk, some = _attention_ref(K, V, q[l, :, h], seen[b], at, kv[b], window, first, sc)
                g = got[l, a:e, h]
                assert (g[~some] == 0).all()
                d = qk * (e_q + (D + 8) * 2.0 ** -24)
                bound = u * np.abs(o) + A * ((1 + u) ** r * np.exp(2 * d)[..., None] - 1) + max(1, len(seen[b])) * 2.0 ** -22 * A
                assert np.isfinite(g).all()
                err = np.abs(g - o)
                assert (err <= bound).all(), (b, l, h, float((err / np.maximum(bound, 1e-300)).max()))
                e2 += float((err ** 2).sum())
                n2 += float((o ** 2).sum())
    lim = np.sqrt(worst) * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17
    assert e2 <= lim * lim * n2, np.sqrt(e2 / n2)
    return out


def _plain(*lens, q=1, body=0):
    return [(n, n - q, q, body) for n in lens]


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("q", [1, 5, 40])
def test_attention_types(dtype, D, q):
    _attention_case(_plain(q, q + 1, 63 + q, 200 + q, 333, q=q), D=D, dtype=dtype)
    _attention_case(_plain(100, 77, q=q), D=D, dtype=dtype, il=True, window=30, first=3, seed=3)


@pytest.mark.parametrize("G,H", [(1, 4), (2, 3), (3, 1), (7, 2), (8, 1), (16, 1), (20, 1)])
@pytest.mark.parametrize("q", [1, 2, 17])
def test_attention_head_layouts(G, H, q):
    _attention_case(_plain(150, 40, q, q=q), G=G, H=H, L=1)
    _attention_case(_plain(150, 96 + q, q=q, body=96), G=G, H=H, L=1, R=32, seed=5)


@pytest.mark.parametrize("R", [1, 5, 16, 20, 48, 64, 128, 300])
@pytest.mark.parametrize("q", [1, 33])
def test_attention_page_sizes(R, q):
    _attention_case(_plain(260, 129, q, q=q), R=R)
    _attention_case(_plain(260, 170, q=q), R=R, window=50, first=7, seed=4)


@pytest.mark.parametrize("q", [1, 3, 12, 70])
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (16, 0), (64, 4), (100, 130), (1000, 5), (37, 1000)])
def test_attention_windows(q, window, first):
    _attention_case(_plain(400, 300, 150, q, q=q), window=window, first=first, R=16, L=1)
    _attention_case([(400, 400 - q, q, 256), (300, 300 - q, q, 64), (160, 160 - q, q, 0)], window=window, first=first, R=32, L=1, seed=9)


@pytest.mark.parametrize("q", [1, 4, 9, 64])
def test_attention_packed(q):
    _attention_case([(200, 200 - q, q, 192), (300, 300 - q, q, 32), (96, 96 - q, q, 96), (130, 130 - q, q, 0), (700, 700 - q, q, 640)], R=64)
    _attention_case([(500, 500 - q, q, 480), (288, 288 - q, q, 288)], R=96, il=True, seed=2)
    _attention_case([(500, 500 - q, q, 480), (288, 288 - q, q, 288)], R=32, G=7, seed=2)


@pytest.mark.parametrize("G,q", [(4, 5), (4, 8), (4, 9), (4, 12), (5, 7), (5, 9), (7, 6), (16, 3), (1, 48), (2, 20), (4, 13), (16, 4)])
def test_packed_rows_for_a_few_parts(G, q):
    """Requests of up to three times 16 query rows that see packed rows keep the accuracy of one of 16, beside
    others that see none, of one token and of more."""
    _attention_case([(200, 200 - q, q, 192), (700, 700 - q, q, 640), (300, 299, 1, 256), (96, 96 - q, q, 96), (90, 90 - q, q, 0),
                     (400, 340, 60, 320)], R=64, L=1, G=G, parts=3)
    _attention_case([(500, 500 - q, q, 480), (300, 300 - q, q, 32), (300, 310, q, 288)], R=32, L=1, G=G, parts=3, window=150, first=5, il=True)


def test_packed_parts_are_captured_and_in_place():
    """A call that takes packed rows in parts uses no scratch: it can be captured, and write over its queries."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R, q = 1, 2, 4, 128, 32, 10
    pool = _pool(L, H, G, D, "bf16")
    t, n = _table([300], R, 3)
    pages = kvr.Pages(_randn(1, (n, L, H, R, D), "bf16"), _randn(2, (n, L, H, R, D), "bf16"))
    packed = pool.packed_pages(n, R)
    pool.page_pack(pages, t, packed, t, [0], [256])
    first = _randn(3, (L, q, H * G, D), "bf16")
    kw = dict(packed=packed, packed_table=t, packed_len=[256])
    want = torch.empty_like(first)
    pool.page_attention(pages, t, [300], [0, q], first, want, **kw)
    x = first.clone()
    torch.cuda.synchronize()
    gc.collect()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.page_attention(pages, t, [300], [0, q], x, x, **kw)
    for _ in range(2):
        x.copy_(first)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    pool.check()


@pytest.mark.parametrize("q", [1, 6, 50])
def test_attention_rows_that_see_nothing(q):
    """An empty cache; queries before it, behind a gap, and with a window that ends before them."""
    _attention_case([(0, 0, q, 0), (0, 90, q, 0), (50, 300, q, 0), (40, 10, q, 0), (1, 0, q, 0)])
    _attention_case([(50, 300, q, 0), (50, 60, q, 0), (0, 5, q, 0), (50, 49, q, 0)], window=20)
    _attention_case([(64, 300, q, 64), (64, 70, q, 32), (50, 300, q, 0)], window=20, first=2, R=32)


@pytest.mark.parametrize("q", [1, 40])
def test_attention_long(q):
    _attention_case(_plain(5000, 9001, q=q), L=1, H=1, R=64)
    _attention_case([(9000, 9000 - q, q, 8960)], L=1, H=1, G=8, R=128, seed=3)
    _attention_case(_plain(9000, q=q), L=1, H=1, R=48, window=4096, first=4)
    _attention_case(_plain(3000, q=q), L=1, H=1, dtype="fp32", D=64)


def test_attention_of_unlike_requests():
    """Single tokens beside prompts and requests without tokens; more requests than fit the parameters."""
    _attention_case([(100, 99, 1, 0), (400, 100, 300, 0), (50, 50, 0, 0), (33, 30, 3, 32), (0, 0, 0, 0), (256, 0, 256, 128)], R=32)
    _attention_case([(30 + i, 29 + i - (i % 5), i % 6, 0) for i in range(140)], L=1, H=1)
    _attention_case([(64 + i, 63 + i, 1, 32 * (i % 3)) for i in range(80)], L=1, R=32)


def test_attention_prompt():
    _attention_case(_plain(700, q=700), L=1, H=1, R=64)
    _attention_case(_plain(900, q=900), L=1, H=2, G=7, R=16, window=200, first=16)
    _attention_case([(1000, 100, 900, 96)], L=1, H=1, R=32, window=130)


def test_attention_scores_that_grow():
    """Large scores, and maxima that move from tile to tile."""
    for q in (1, 40):
        _attention_case(_plain(700, 300, q=q), spread=3.0, L=1)
        _attention_case([(700, 700 - q, q, 640)], spread=3.0, L=1, R=64)
        _attention_case(_plain(300, q=q), scale=0.9, L=1)


def test_attention_default_positions_and_in_place():
    for q in (1, 3, 30):
        _attention_case(_plain(80, 60, q=q), default_pos=True, in_place=True)
        _attention_case(_plain(80, 60, q=q), in_place=True, D=64, dtype="fp32")


@pytest.mark.parametrize("q", [1, 20, 50])
def test_attention_over_padded_pages(q):
    _attention_case(_plain(300, 170, q=q), pad=8, R=16, L=2)
    _attention_case(_plain(300, 170, q=q), pad=256, R=64, L=2, window=90, first=5)
    _attention_case([(300, 300 - q, q, 256), (90, 90 - q, q, 32)], pad=24, R=32, L=2)
    _attention_case(_plain(200, q=q), pad=8, R=20, dtype="fp32", D=64)


def test_attention_of_one_and_two_tiles_of_rows():
    """Blocks of up to 128 rows beside larger ones, and alone; both orders."""
    for R in (16, 20):
        _attention_case(_plain(300, q=20) + _plain(400, q=40) + _plain(500, q=64) + _plain(260, q=33) + _plain(90, q=70), R=R, L=1)
        _attention_case(_plain(300, q=20) + _plain(1400, q=32) + _plain(130, q=5) + _plain(31, q=31), R=R, L=3, H=2)
    _attention_case([(300, 236, 64, 288), (700, 620, 80, 32), (40, 20, 20, 32)], R=32, L=1, window=150, first=10)


@pytest.mark.parametrize("R", [16, 32, 48, 64, 128, 256, 20])
def test_first_rows_and_window_in_one_tile(R):
    """First rows that fill a part of a 128-row tile, whose rest is the window's: by boxes of 16 to 64 rows
    and by hand; blocks of one and of two tiles, cut in stretches too."""
    for first, window in ((4, 100), (40, 64), (64, 300), (70, 33), (129, 257)):
        _attention_case(_plain(900, 515, q=70), R=R, L=1, H=1, window=window, first=first)
        _attention_case(_plain(700, q=20) + _plain(390, q=32), R=R, L=1, H=1, window=window, first=first, seed=6)
    _attention_case(_plain(5000, q=40), R=R, L=1, H=1, window=4000, first=5)
    if R % 32 == 0:
        _attention_case([(900, 830, 70, 512), (900, 830, 70, 32), (900, 830, 70, 0)], R=R, L=1, H=1, window=300, first=40)


def test_outputs_at_16_bytes():
    """Rows of an output that starts 16 bytes behind a 32-byte boundary, for both kernels."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R = 1, 2, 4, 128, 32
    pool = _pool(L, H, G, D, "bf16")
    t, n = _table([300, 90], R, 3)
    pages = kvr.Pages(_randn(1, (n, L, H, R, D), "bf16"), _randn(2, (n, L, H, R, D), "bf16"))
    for lq in ((70, 40), (1, 3)):
        T = sum(lq)
        q = _randn(3, (L, T, H * G, D), "bf16")
        outs = []
        for off in (0, 8):
            buf = torch.zeros(q.numel() + 16, device="cuda", dtype=q.dtype)
            out = buf[off:off + q.numel()].view(q.shape)
            assert out.data_ptr() % 32 == 2 * off
            pool.page_attention(pages, t, [300, 90], _starts(lq).astype(np.int32), q, out)
            torch.cuda.synchronize()
            pool.check()
            assert not buf[:off].any() and not buf[off + q.numel():].any()
            outs.append(out)
        assert torch.equal(*outs) and outs[0].any()


def test_attention_is_deterministic_and_leaves_the_cache():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    for reqs in (_plain(2000, 77), _plain(2000, 300, q=40), [(1500, 1470, 30, 1472), (900, 899, 1, 864)]):
        a = _attention_case(reqs, R=32, seed=7)
        for _ in range(3):
            assert torch.equal(a, _attention_case(reqs, R=32, seed=7, twice=True))
    pool = _pool(2, 2, 4, 128, "bf16")
    k, v = _randn(1, (9, 2, 2, 16, 128), "bf16"), _randn(2, (9, 2, 2, 16, 128), "bf16")
    k0, v0 = k.clone(), v.clone()
    for q in (1, 30):
        Q = _randn(3, (2, q, 8, 128), "bf16")
        pool.page_attention(kvr.Pages(k, v), [list(range(9))], [130], [0, q], Q, torch.empty_like(Q))
    torch.cuda.synchronize()
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_requests_that_share_pages():
    """Two requests on one prefix's pages, each with its own last page: as each alone."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R = 2, 2, 4, 128, 32
    pool = _pool(L, H, G, D, "bf16")
    pages = kvr.Pages(_randn(1, (8, L, H, R, D), "bf16"), _randn(2, (8, L, H, R, D), "bf16"))
    t = [[5, 2, 0, 7, 4], [5, 2, 0, 1, 3]]
    for q in (1, 3, 30):
        Q = _randn(3, (L, 2 * q, H * G, D), "bf16")
        both, alone = torch.empty_like(Q), torch.empty_like(Q)
        pool.page_attention(pages, t, [110, 99 + q], [0, q, 2 * q], Q, both)
        for b, n in enumerate((110, 99 + q)):
            o = torch.empty((L, q, H * G, D), device="cuda", dtype=torch.bfloat16)
            pool.page_attention(pages, [t[b]], [n], [0, q], Q[:, b * q:(b + 1) * q].contiguous(), o)
            alone[:, b * q:(b + 1) * q] = o
        torch.cuda.synchronize()
        d = (both.double() - alone.double()).norm() / alone.double().norm()
        assert d <= np.sqrt(2 * 3) * 2.0 ** -8, float(d)


def test_restored_rows_in_slices():
    """Packed rows that the scratch holds in two slices of the units only: bit for bit what their
    unpacked pages give, which meet the same products."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R, n = 9, 8, 1, 128, 128, 33152
    pool = _pool(L, H, G, D, "bf16")
    k, v = (_randn(i, (n // R, L, H, R, D), "bf16") for i in (1, 2))
    t = np.random.default_rng(0).permutation(n // R).astype(np.int32)[None]
    packed = pool.packed_pages(n // R, R)
    pool.page_pack(kvr.Pages(k, v), t, packed, t, [0], [n])
    pool.page_unpack(packed, t, kvr.Pages(k, v), t, [0], [n])
    Q = _randn(3, (L, 40, H * G, D), "bf16")
    a, b = torch.empty_like(Q), torch.empty_like(Q)
    pool.page_attention(kvr.Pages(k, v), t, [n], [0, 40], Q, a, packed=packed, packed_table=t, packed_len=[n])
    pool.page_attention(kvr.Pages(k, v), t, [n], [0, 40], Q, b)
    torch.cuda.synchronize()
    pool.check()
    # (another number of stretches may be taken: the order of sums)
    d = (a.double() - b.double()).norm() / b.double().norm()
    assert d <= np.sqrt(2 * 3) * 2.0 ** -8, float(d)
    assert (a.view(-1, D).double() - b.view(-1, D).double()).norm(dim=1).max() <= 2.0 ** -5 * b.double().view(-1, D).norm(dim=1).max()


def test_pages_beyond_32_bit_offsets():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R = 2, 2, 4, 128, 128
    n = (1 << 31) // (L * H * R * D) + 40                     # elements of k alone pass 2^31
    pool = _pool(L, H, G, D, "bf16")
    k, v = (torch.empty((n, L, H, R, D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    packed = kvr.PackedPages(torch.empty(((1 << 32) // pool.packed_page_bytes(R) + 40, pool.packed_page_bytes(R)), device="cuda", dtype=torch.uint8), R)
    small = [_randn(i, (3, L, H, R, D), "bf16") for i in (1, 2)]
    hi = [n - 1, n - 30, n - 2]
    for x, y in zip((k, v), small):
        for i, p in enumerate(hi):
            x[p] = y[i]
    far, near = kvr.Pages(k, v), kvr.Pages(*small)
    tp = [[packed.data.shape[0] - 1, packed.data.shape[0] - 20, packed.data.shape[0] - 3]]
    near_packed = pool.packed_pages(3, R)
    nk, nv = _randn(5, (L, 70, H, D), "bf16"), _randn(6, (L, 70, H, D), "bf16")
    for pages, t, pk, pt in ((far, [hi], packed, tp), (near, [[0, 1, 2]], near_packed, [[0, 1, 2]])):
        pool.page_append(pages, t, [300], [0, 70], nk, nv)
        pool.page_pack(pages, t, pk, pt, [0], [256])
    for q in (1, 4, 40):
        Q = _randn(7, (L, q, H * G, D), "bf16")
        o = [torch.empty_like(Q) for _ in range(4)]
        pool.page_attention(far, [hi], [370], [0, q], Q, o[0])
        pool.page_attention(near, [[0, 1, 2]], [370], [0, q], Q, o[1])
        pool.page_attention(far, [hi], [370], [0, q], Q, o[2], packed=packed, packed_table=tp, packed_len=[256])
        pool.page_attention(near, [[0, 1, 2]], [370], [0, q], Q, o[3], packed=near_packed, packed_table=[[0, 1, 2]], packed_len=[256])
        torch.cuda.synchronize()
        pool.check()
        assert torch.equal(o[0], o[1]) and torch.equal(o[2], o[3]) and not torch.equal(o[0], o[2])
    u = [torch.zeros_like(x) for x in small]
    pool.page_unpack(packed, tp, kvr.Pages(*u), [[0, 1, 2]], [0], [256])
    w = [torch.zeros_like(x) for x in small]
    pool.page_unpack(near_packed, [[0, 1, 2]], kvr.Pages(*w), [[0, 1, 2]], [0], [256])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(u, w))


def test_streams_and_graphs():
    """A decode step (append, attention, the packing of a full page) captured once and replayed on
    new inputs, on two streams at once; what needs scratch or uploads is refused in a capture."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R, n = 2, 2, 4, 128, 32, 129
    pool = _pool(L, H, G, D, "bf16")
    pool.reserve(max_batch=128, max_spans=4096, max_query_tokens=256)
    t, tp = [[0, 1, 2, 3, 4]], [[0, 1, 2, 3]]

    def state(seed):
        k, v = _randn(seed, (5, L, H, R, D), "bf16"), _randn(seed + 1, (5, L, H, R, D), "bf16")
        s = dict(k=k, v=v, pages=kvr.Pages(k, v), packed=pool.packed_pages(4, R), q=_randn(seed + 2, (L, 1, H * G, D), "bf16"),
                 nk=_randn(seed + 3, (L, 1, H, D), "bf16"), nv=_randn(seed + 4, (L, 1, H, D), "bf16"))
        s["out"] = torch.empty_like(s["q"])
        return s

    gc.collect()      # (an older test's pool that is released during a capture ends the capture)

    def step(s):
        pool.page_append(s["pages"], t, [n - 1], [0, 1], s["nk"], s["nv"])
        pool.page_pack(s["pages"], t, s["packed"], tp, [0], [128])
        pool.page_attention(s["pages"], t, [n], [0, 1], s["q"], s["out"], packed=s["packed"], packed_table=tp, packed_len=[128],
                            window=100, n_first=3)

    states, graphs, streams = [state(10), state(20)], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, st in zip(states, streams):
        with torch.cuda.stream(st):
            step(s)                       # warm
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step(s)
        graphs.append(g)
    for seed in (30, 50):
        fresh = [state(seed), state(seed + 10)]
        want = []
        for s, f in zip(states, fresh):
            for x in ("k", "v", "q", "nk", "nv"):
                s[x].copy_(f[x])
            step(f)
            want.append(f["out"])
        torch.cuda.synchronize()
        for _ in range(20):               # both at once
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            assert torch.equal(s["out"], w)
    pool.check()

    def refused(call):
        """... and the capture stays usable."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            states[0]["out"].zero_()
            with pytest.raises(kvr.KvrError) as e:
                call()
        assert e.value.status == 3
        g.replay()
        torch.cuda.synchronize()
        assert (states[0]["out"] == 0).all()

    s, Q = states[0], _randn(1, (L, 20, H * G, D), "bf16")
    refused(lambda: pool.page_attention(s["pages"], t, [n], [0, 20], Q, Q))
    many = [[i % 5] for i in range(70)]
    Q70 = _randn(1, (L, 70, H * G, D), "bf16")
    refused(lambda: pool.page_attention(s["pages"], many, [20] * 70, list(range(71)), Q70, Q70))
    step(s)                               # and all goes on
    pool.page_attention(s["pages"], t, [n], [0, 20], Q, Q)
    torch.cuda.synchronize()
    pool.check()


def test_calls_on_several_streams_share_the_scratch_in_turn():
    """Query prefills of one pool on two streams, enqueued alternately."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R = 2, 2, 4, 128, 32
    pool = _pool(L, H, G, D, "bf16")
    jobs = []
    for i in range(6):
        n, q = 400 + 77 * i, 20 + 9 * i
        k, v = _randn(10 * i, (30, L, H, R, D), "bf16"), _randn(10 * i + 1, (30, L, H, R, D), "bf16")
        Q = _randn(10 * i + 2, (L, q, H * G, D), "bf16")
        jobs.append((kvr.Pages(k, v), [list(range(30))], [n], [0, q], Q, torch.empty_like(Q), torch.empty_like(Q), pool.packed_pages(30, R)))
    torch.cuda.synchronize()
    for pages, t, n, qo, Q, o, w, pk in jobs:
        pool.page_pack(pages, t, pk, t, [0], [320])
        pool.page_attention(pages, t, n, qo, Q, w, packed=pk, packed_table=t, packed_len=[320])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, (pages, t, n, qo, Q, o, w, pk) in enumerate(jobs * 3):
        pool.page_attention(pages, t, n, qo, Q, o, packed=pk, packed_table=t, packed_len=[320], stream=streams[i % 2])
    torch.cuda.synchronize()
    pool.check()
    assert all(torch.equal(o, w) for *_, o, w, _ in jobs)


def test_bad_queries_are_reported_and_only_they():
    import torch
    from rag_precomputed_kv_gb300 import kvr
    for dtype, D in (("bf16", 128), ("fp32", 64)):
        pool = _pool(1, 1, 4, D, dtype)
        pages = kvr.Pages(_randn(1, (4, 1, 1, 32, D), dtype), _randn(2, (4, 1, 1, 32, D), dtype))
        t = [[0, 1], [2, 3]]
        for q in (1, 30):
            Q = _randn(3, (1, 2 * q, 4, D), dtype)
            good = torch.empty_like(Q)
            args = (pages, t, [60, 30 + q], [0, q, 2 * q])
            kw = dict(q_pos=[60 - q, 30])
            pool.page_attention(*args, Q, good, **kw)
            torch.cuda.synchronize()
            pool.check()
            Q[0, 0, 1, 5] = float("nan")
            bad = torch.empty_like(Q)
            pool.page_attention(*args, Q, bad, **kw)
            with pytest.raises(kvr.KvrError) as e:
                pool.check()
            assert e.value.status == 6
            same = (bad == good).all(-1)
            same[0, 0, 1] = True
            assert same.all() and not torch.isfinite(bad[0, 0, 1]).any()
            # a query of NaN that sees nothing gives zeros, and no error
            pool.page_attention(pages, t, [0, 0], [0, q, 2 * q], Q, bad, q_pos=[5, 9])
            torch.cuda.synchronize()
            pool.check()
            assert (bad == 0).all()


def test_a_cache_as_it_is_used():
    """A stitched prefix goes to pages, the query is appended and attends as over the flat cache;
    full pages are packed, decode steps follow, with a window at the end."""
    import torch
    from rag_precomputed_kv_gb300 import kvr
    L, H, G, D, R = 2, 2, 4, 128, 64
    k, v = _randn(1, (6, L, H, 100, D), "bf16"), _randn(2, (6, L, H, 100, D), "bf16")
    pool = kvr.Pool(k, v, H * G, THETA)
    P, lq = 290, 30
    co, qo = [0, P + lq], [0, lq]
    ck, cv = (torch.zeros((co[-1] * L * H, D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    Q, KQ, VQ = _randn(3, (L, lq, H * G, D), "bf16"), _randn(4, (L, lq, H, D), "bf16"), _randn(5, (L, lq, H, D), "bf16")
    out, flat = torch.empty_like(Q), torch.empty_like(Q)
    plen = pool.assemble([0, 3], [(0, 0, 100), (3, 10, 100), (5, 0, 100)], co, ck, cv)
    assert plen.tolist() == [P]
    pk, pv = (torch.full((8, L, H, R, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pages, table = kvr.Pages(pk, pv), torch.tensor([[6, 1, 4, 0, 7, 3, 2]], dtype=torch.int32)
    blocks = [x.view(L, H, P + lq, D)[:, :, :P].transpose(1, 2) for x in (ck, cv)]
    pool.page_append(pages, table, [0], [0, P], *blocks, turned=True)
    pool.page_append(pages, table, [P], qo, KQ, VQ)
    pool.page_attention(pages, table, [P + lq], qo, Q, out)
    pool.query_attention(co, plen, qo, Q, KQ, VQ, ck, cv, flat)
    torch.cuda.synchronize()
    pool.check()
    rows = torch.arange(P + lq)
    ids = table[0, rows // R].long().cuda()
    assert torch.equal(pk[ids, :, :, (rows % R).cuda()].permute(1, 2, 0, 3), ck.view(L, H, P + lq, D))
    # both round the same queries and probabilities, in another order of sums
    d = (out.double() - flat.double()).norm() / flat.double().norm()
    assert d <= np.sqrt(2 * 4) * 2.0 ** -8, float(d)
    # decode: the full pages in 4 bits, their bf16 pages given away
    packed = pool.packed_pages(5, R)
    pool.page_pack(pages, table, packed, [[0, 1, 2, 3, 4]], [0], [256])
    u = [torch.zeros_like(pk), torch.zeros_like(pv)]
    pool.page_unpack(packed, [[0, 1, 2, 3]], kvr.Pages(*u), table, [0], [256])
    n = P + lq
    for step in range(3):
        q1, k1, v1 = _randn(10 + step, (L, 1, H * G, D), "bf16"), _randn(20 + step, (L, 1, H, D), "bf16"), _randn(30 + step, (L, 1, H, D), "bf16")
        pool.page_append(pages, table, [n], [0, 1], k1, v1)
        n += 1
        o1, o2 = torch.empty_like(q1), torch.empty_like(q1)
        rest = table.clone()
        rest[0, :4] = -1
        kw = dict(window=200, n_first=2) if step == 2 else {}
        pool.page_attention(pages, rest, [n], [0, 1], q1, o1, packed=packed, packed_table=[[0, 1, 2, 3]], packed_len=[256], **kw)
        for x, y in zip(u, (pk, pv)):       # the same rows, restored to bf16
            for g in range(4, 7):
                x[int(table[0, g])] = y[int(table[0, g])]
        pool.page_attention(kvr.Pages(*u), table, [n], [0, 1], q1, o2, **kw)
        torch.cuda.synchronize()
        pool.check()
        d = (o1.double() - o2.double()).norm() / o2.double().norm()
        assert d <= np.sqrt(2 * 5) * 2.0 ** -8, float(d)   # (keys and values of o2 rounded once more)
