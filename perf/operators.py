"""Measured cases of the cache operators: query attention over a prefix shared
by a group of requests, the attention weight that a cache's keys accumulate,
and the eviction of a cache's lightest rows.

Layouts are the library's: a cache is flat, request b's block holding R_b rows
per (layer, kv-head) from row ``offsets[b] * L * H_kv`` on, inside it
``[L][H_kv][R_b][D]``; queries are ``[L][T][H_q][D]``, not rotated; RoPE pairs
are (x_i, x_i+D/2).
"""
import math

import torch

own = False

# layers, query heads, kv heads, head dim, RoPE base of the served models
QWEN2_7B = dict(layers=28, q_heads=28, kv_heads=4, dim=128, theta=1e6, dtype="bf16")
QWEN3_8B = dict(layers=36, q_heads=32, kv_heads=8, dim=128, theta=1e6, dtype="bf16")
LLAMA31_8B = dict(layers=32, q_heads=32, kv_heads=8, dim=128, theta=5e5, dtype="bf16")
TINY = dict(layers=1, q_heads=4, kv_heads=2, dim=64, theta=1e4, dtype="fp32")


def listed():
    return [
        # four users ask about the same five retrieved chunks; a decode step
        dict(QWEN2_7B, name="shared-decode-4", op="shared", groups=1, per_group=4, prefix=2592, own=96, spread=63, q=1),
        # a serving batch on one long system prompt with tools and few-shot examples
        dict(QWEN3_8B, name="shared-decode-64", op="shared", groups=1, per_group=64, prefix=8256, own=128, spread=96, q=1),
        # sixteen sessions over the same 32k-token document set
        dict(LLAMA31_8B, name="shared-decode-32k", op="shared", groups=1, per_group=16, prefix=33248, own=64, spread=31, q=1),
        # two sets of retrieved chunks, eight questions on each: their prefill
        dict(QWEN2_7B, name="shared-prefill", op="shared", groups=2, per_group=8, prefix=2592, own=0, spread=15, q=64),
        # the small fp32 configuration
        dict(TINY, name="shared-tiny", op="shared", groups=1, per_group=3, prefix=193, own=5, spread=4, q=1),
        # weights of one decode step over one request's stitched cache
        dict(QWEN2_7B, name="weights-decode", op="weights", batch=1, prefix=2656, spread=0, q=1, add=True),
        # the last 32 query tokens of each request of a serving batch look back
        dict(QWEN3_8B, name="weights-window", op="weights", batch=16, prefix=1216, spread=300, q=32, add=False),
        # a decode step over two 32k-token document caches
        dict(LLAMA31_8B, name="weights-32k", op="weights", batch=2, prefix=33280, spread=64, q=1, add=True),
        # the small fp32 configuration
        dict(TINY, name="weights-tiny", op="weights", batch=1, prefix=203, spread=0, q=16, add=False),
        # one request's cache cut to a budget after its prefill
        dict(QWEN2_7B, name="evict-one", op="evict", batch=1, rows=2656, spread=0, keep=1024, first=32, recent=64),
        # a serving batch cut to 512 rows a request
        dict(QWEN3_8B, name="evict-batch", op="evict", batch=16, rows=1344, spread=300, keep=512, first=64, recent=128),
        # a 32k-token cache cut to an eighth
        dict(LLAMA31_8B, name="evict-32k", op="evict", batch=1, rows=33504, spread=0, keep=4096, first=4, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("shared", "weights", "evict"))
    m = dict(rng.choice((QWEN2_7B, QWEN3_8B, LLAMA31_8B, QWEN2_7B, QWEN3_8B, LLAMA31_8B, TINY)))
    m["layers"] = rng.randint(1, m["layers"])
    if m["dim"] == 64:
        m["dtype"] = rng.choice(("fp32", "bf16"))
    tiny = m["dim"] == 64
    units = m["layers"] * m["kv_heads"]
    top = 2000 if tiny else 33000
    if op == "shared":
        groups, per_group = rng.randint(1, 3), _log(rng, 1, 4 if tiny else 32)
        q = rng.choice((1, 1, 1, rng.randint(2, 80)))
        prefix = _log(rng, 40, min(top, max(64, 220 * 33248 // (units * groups))))
        # keep the products and the plain form's scores within the largest listed case
        while groups * per_group * q * prefix > 64 * 8256 * 2.7:
            q = max(1, q // 2)
            prefix = max(40, prefix // 2)
        return dict(m, op=op, groups=groups, per_group=per_group, prefix=prefix, own=rng.randint(0, 160),
                    spread=rng.randint(0, 40), q=q)
    batch = _log(rng, 1, 3 if tiny else 16)
    rows = _log(rng, 60, min(top, max(64, 2 * 256 * 33280 // (units * batch) // (4 if op == "evict" else 1))))
    if op == "weights":
        q = rng.choice((1, 1, rng.randint(2, 64)))
        while batch * q * rows > 16 * 32 * 1500:
            q = max(1, q // 2)
            rows = max(60, rows // 2)
        return dict(m, op=op, batch=batch, prefix=rows, spread=rng.randint(0, rows // 2), q=q,
                    add=rng.choice((True, False)))
    first, recent = rng.randint(0, 8), rng.randint(0, 20)
    return dict(m, op=op, batch=batch, rows=rows, spread=rng.randint(0, rows // 2),
                keep=rng.randint(first + recent + 1, rows), first=first, recent=recent)


# ---- sizes of a case ----
def _ragged(base, spread, n):
    """n lengths in [base - spread, base], from the case alone."""
    return [base - (i * 7919) % (spread + 1) for i in range(n)]


def _starts(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _shared_sizes(c):
    B = c["groups"] * c["per_group"]
    prefix = _ragged(c["prefix"], 30, c["groups"])
    own_rows = [max(0, n) for n in _ragged(c["own"], min(c["spread"], c["own"]), B)]
    q = _ragged(c["q"], min(c["spread"], c["q"] - 1), B)
    return B, prefix, own_rows, q


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    D, L, Hq, H = c["dim"], c["layers"], c["q_heads"], c["kv_heads"]
    row = L * H * D * e            # one token's keys (or values) in every layer and kv head
    if c["op"] == "shared":
        B, prefix, own_rows, q = _shared_sizes(c)
        T = sum(q)
        pairs = sum(q[b] * prefix[b // c["per_group"]] + q[b] * own_rows[b] + q[b] * (q[b] + 1) // 2 for b in range(B))
        # the prefix and the own rows once, queries in and out, the new keys and values in and appended
        return {"bytes": 2 * row * (sum(prefix) + sum(own_rows) + 2 * T) + 2 * T * L * Hq * D * e,
                "flops": 4 * D * Hq * L * pairs}
    if c["op"] == "weights":
        P = _ragged(c["prefix"], c["spread"], c["batch"])
        n = sum(P) + c["q"] * c["batch"]
        pairs = sum(c["q"] * p + c["q"] * (c["q"] + 1) // 2 for p in P)
        return {"bytes": row * n + c["batch"] * c["q"] * L * Hq * D * e + L * H * n * 4 * (2 if c["add"] else 1),
                "flops": 2 * D * Hq * L * pairs}
    n = _ragged(c["rows"], c["spread"], c["batch"])
    kept = sum(min(c["keep"], x) for x in n)
    # the weights in, the kept rows in and out, their indexes and weights out
    return {"bytes": 4 * L * H * sum(n) + 4 * row * kept + 8 * L * H * kept, "flops": 3 * D * L * H * kept}


# ---- inputs ----
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(c):
    """The handle a program keeps: a pool of this layout (its chunks are not read here)."""
    from rag_precomputed_kv_gb300 import kvr
    k = torch.zeros((1, c["layers"], c["kv_heads"], 8, c["dim"]), device="cuda", dtype=_dtype(c))
    return kvr.Pool(k, torch.zeros_like(k), c["q_heads"], c["theta"])


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c, g, dt = case, _gen(seed), _dtype(case)
    D, L, Hq, H = c["dim"], c["layers"], c["q_heads"], c["kv_heads"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    s = {"case": c}
    if own:
        s["pool"] = _pool(c)
    if c["op"] == "shared":
        B, prefix, own_rows, q = _shared_sizes(c)
        T = sum(q)
        cap = [own_rows[b] + q[b] + 3 for b in range(B)]           # room for the next tokens
        s.update(group_offsets=_starts([c["per_group"]] * c["groups"]), prefix_offsets=_starts(prefix), prefix_len=prefix,
                 cache_offsets=_starts(cap), own_len=own_rows, q_offsets=_starts(q),
                 prefix_k=randn(sum(prefix) * L * H, D), prefix_v=randn(sum(prefix) * L * H, D),
                 cache_k=randn(sum(cap) * L * H, D), cache_v=randn(sum(cap) * L * H, D),
                 q=randn(L, T, Hq, D), kq=randn(L, T, H, D), vq=randn(L, T, H, D),
                 out=torch.zeros((L, T, Hq, D), device="cuda", dtype=dt))
    elif c["op"] == "weights":
        P = _ragged(c["prefix"], c["spread"], c["batch"])
        rows = [p + c["q"] + 5 for p in P]
        s.update(cache_offsets=_starts(rows), prefix_len=P, q_offsets=_starts([c["q"]] * c["batch"]),
                 q=randn(L, c["batch"] * c["q"], Hq, D), cache_k=randn(sum(rows) * L * H, D),
                 weights=torch.rand(sum(rows) * L * H, generator=g, device="cuda") * (1e-3 if c["add"] else 0.0))
    else:
        n = _ragged(c["rows"], c["spread"], c["batch"])
        rows = [x + 8 for x in n]
        kept = [min(c["keep"], x) for x in n]
        dst = [x + 32 for x in kept]                               # the budget and room to decode
        # accumulated attention weight: few heavy rows, a long tail
        w = torch.exp(2.5 * torch.randn(sum(rows) * L * H, generator=g, device="cuda")) / max(n)
        s.update(cache_offsets=_starts(rows), kv_len=n, keep=[c["keep"]] * c["batch"], dst_offsets=_starts(dst), weights=w,
                 cache_k=randn(sum(rows) * L * H, D), cache_v=randn(sum(rows) * L * H, D),
                 dst_k=torch.zeros((sum(dst) * L * H, D), device="cuda", dtype=dt),
                 dst_v=torch.zeros((sum(dst) * L * H, D), device="cuda", dtype=dt),
                 dst_weights=torch.zeros(sum(dst) * L * H, device="cuda"),
                 kept=torch.zeros(sum(kept) * L * H, device="cuda", dtype=torch.int32))
    return s


# ---- one pass ----
def run(state):
    s, c = state, state["case"]
    if c["op"] == "shared":
        if own:
            s["pool"].shared_query_attention(s["group_offsets"], s["prefix_offsets"], s["prefix_len"], s["prefix_k"],
                                             s["prefix_v"], s["cache_offsets"], s["own_len"], s["q_offsets"], s["q"],
                                             s["kq"], s["vq"], s["cache_k"], s["cache_v"], s["out"])
        else:
            _plain_shared(s, c)
        return {"out": s["out"], "cache_k": s["cache_k"], "cache_v": s["cache_v"]}
    if c["op"] == "weights":
        if own:
            s["pool"].key_weights(s["cache_offsets"], s["prefix_len"], s["q_offsets"], s["q"], s["cache_k"], s["weights"],
                                  accumulate=c["add"])
        else:
            _plain_weights(s, c)
        return {"weights": s["weights"]}
    if own:
        s["pool"].evict(s["cache_offsets"], s["kv_len"], s["keep"], s["weights"], s["cache_k"], s["cache_v"], s["kept"],
                        dst_offsets=s["dst_offsets"], dst_k=s["dst_k"], dst_v=s["dst_v"], dst_weights=s["dst_weights"],
                        n_first=c["first"], n_recent=c["recent"])
    else:
        _plain_evict(s, c)
    return {"kept": s["kept"], "dst_k": s["dst_k"], "dst_v": s["dst_v"], "dst_weights": s["dst_weights"]}


# ---- the plain forms ----
def _dev(x):
    return torch.tensor(x, device="cuda", dtype=torch.int64)


def _turn(x, pos, theta):
    """x [..., D] in fp32 turned by pos [...]; the angles in 64 bits."""
    h = x.shape[-1] // 2
    w = theta ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    a = pos[..., None].double() * w
    co, si = torch.cos(a).float(), torch.sin(a).float()
    lo, hi = x[..., :h], x[..., h:]
    return torch.cat([lo * co - hi * si, lo * si + hi * co], -1)


def _block_rows(offsets, units, n_rows):
    """Flat row of (request, unit, row): [B, units, n_rows], rows past a block clamped to its last one."""
    o = _dev(offsets)
    cap = o[1:] - o[:-1]
    j = torch.minimum(torch.arange(n_rows, device="cuda")[None, :], cap[:, None] - 1).clamp_min(0)
    u = torch.arange(units, device="cuda")
    return o[:-1, None, None] * units + u[None, :, None] * cap[:, None, None] + j[:, None, :]


def _tokens(q_offsets):
    """Per request and padded token: the token's index; per token: its request and place."""
    o = _dev(q_offsets)
    n = o[1:] - o[:-1]
    t = torch.arange(int(max(b - a for a, b in zip(q_offsets, q_offsets[1:]))), device="cuda")
    tok = torch.minimum(o[:-1, None] + t[None, :], o[-1] - 1)
    b_of = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    return tok, b_of, torch.arange(int(q_offsets[-1]), device="cuda") - o[b_of]


def _query_rows(q, tok, pos, c):
    """q [L, T, Hq, D] -> [B, L * H, tokens * G, D], turned by pos [B, tokens]."""
    L, _, Hq, D = q.shape
    H, (B, n) = c["kv_heads"], tok.shape
    x = _turn(q[:, tok].float(), pos[None, :, :, None], c["theta"])            # [L, B, n, Hq, D]
    return x.view(L, B, n, H, Hq // H, D).permute(1, 0, 3, 2, 4, 5).reshape(B, L * H, n * (Hq // H), D)


def _plain_shared(s, c):
    L, H, D, G = c["layers"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    U, B, scale = L * H, len(s["own_len"]), 1.0 / math.sqrt(c["dim"])
    per = c["per_group"]
    tok, b_of, t_of = _tokens(s["q_offsets"])
    n_tok = tok.shape[1]
    plen, olen = _dev(s["prefix_len"]), _dev(s["own_len"])
    pos = plen.repeat_interleave(per)[:, None] + olen[:, None] + torch.arange(n_tok, device="cuda")   # [B, n]
    # append the query tokens' keys (turned) and values
    n_own = max(a + b - o for a, b, o in zip(s["own_len"], s["q_offsets"][1:], s["q_offsets"]))
    row_of = _block_rows(s["cache_offsets"], U, n_own)
    at = row_of[b_of, :, (olen[b_of] + t_of)].T.reshape(L, H, -1).transpose(1, 2)             # [L, T, H]
    s["cache_k"][at] = _turn(s["kq"].float(), pos[b_of, t_of][None, :, None], c["theta"]).to(s["cache_k"].dtype)
    s["cache_v"][at] = s["vq"]
    q = _query_rows(s["q"], tok, pos, c)                                                      # [B, U, n * G, D]
    # the shared prefix, for all requests of a group at once
    n_pre = max(s["prefix_len"])
    pre = _block_rows(s["prefix_offsets"], U, n_pre)
    qg = q.view(c["groups"], per, U, -1, D).transpose(1, 2).reshape(c["groups"], U, -1, D)
    sp = qg @ s["prefix_k"][pre].float().transpose(-1, -2) * scale
    sp.masked_fill_((torch.arange(n_pre, device="cuda") >= plen[:, None])[:, None, None, :], -math.inf)
    sp = sp.view(c["groups"], U, per, n_tok * G, n_pre)
    # each request's own rows, causal
    so = q @ s["cache_k"][row_of].float().transpose(-1, -2) * scale
    last = olen[:, None] + torch.arange(n_tok, device="cuda")
    hidden = torch.arange(n_own, device="cuda") > last.repeat_interleave(G, 1)[:, :, None]
    so.masked_fill_(hidden[:, None], -math.inf)
    so = so.view(c["groups"], per, U, n_tok * G, n_own).transpose(1, 2)
    m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
    sp = torch.exp(sp.sub_(m))
    so = torch.exp(so.sub_(m))
    z = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    vo = s["cache_v"][row_of].float().masked_fill((torch.arange(n_own, device="cuda") >= (last[:, -1:] + 1))[:, None, :, None], 0.0)
    o = (sp.view(c["groups"], U, -1, n_pre) @ s["prefix_v"][pre].float()).view(c["groups"], U, per, n_tok * G, D)
    o = o.add_(so @ vo.view(c["groups"], per, U, n_own, D).transpose(1, 2)).div_(z)
    o = o.transpose(1, 2).reshape(B, L, H, n_tok, G, D)[b_of, :, :, t_of]                     # [T, L, H, G, D]
    s["out"].copy_(o.transpose(0, 1).reshape(s["out"].shape))


def _plain_weights(s, c):
    L, H, G = c["layers"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    U = L * H
    tok, b_of, t_of = _tokens(s["q_offsets"])
    n_tok, P = tok.shape[1], _dev(s["prefix_len"])
    pos = P[:, None] + torch.arange(n_tok, device="cuda")
    q = _query_rows(s["q"], tok, pos, c)
    n = max(s["prefix_len"]) + n_tok
    rows = _block_rows(s["cache_offsets"], U, n)
    sc = q @ s["cache_k"][rows].float().transpose(-1, -2) * (1.0 / math.sqrt(c["dim"]))
    j = torch.arange(n, device="cuda")
    sc.masked_fill_((j > pos.repeat_interleave(G, 1)[:, :, None])[:, None], -math.inf)
    sc = torch.exp(sc.sub_(sc.amax(-1, keepdim=True)))
    w = (sc / sc.sum(-1, keepdim=True)).sum(2)                                                 # [B, U, n]
    keys = (j < P[:, None] + n_tok)[:, None].expand_as(w)
    old = s["weights"][rows[keys]] if c["add"] else 0.0
    s["weights"][rows[keys]] = w[keys] + old


def _plain_evict(s, c):
    U, n_max = c["layers"] * c["kv_heads"], max(s["kv_len"])
    n = _dev(s["kv_len"])[:, None, None]
    kk = torch.minimum(_dev(s["keep"])[:, None, None], n)
    src = _block_rows(s["cache_offsets"], U, n_max)
    j = torch.arange(n_max, device="cuda")
    w = s["weights"][src]
    w = torch.where((j < c["first"]) | (j >= n - c["recent"]), math.inf, w)
    w = torch.where(j >= n, -math.inf, w)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    k_max = min(max(s["keep"]), n_max)
    i = torch.arange(k_max, device="cuda")
    mine = (i < kk).expand(-1, U, -1)
    kept = torch.sort(torch.where(mine, order[..., :k_max], n_max), dim=-1).values
    s["kept"].copy_(kept[mine])
    kept = kept.clamp_max(n_max - 1)
    frm = torch.gather(src, 2, kept)[mine]
    to = _block_rows(s["dst_offsets"], U, k_max)[mine]
    turned = _turn(s["cache_k"][frm].float(), (i - kept)[mine], c["theta"])
    s["dst_k"][to] = turned.to(s["dst_k"].dtype)
    s["dst_v"][to] = s["cache_v"][frm]
    s["dst_weights"].zero_()
    s["dst_weights"][to] = s["weights"][frm]


# ---- the definitions in 64 bits, request by request ----
def _angle64(n, pos, theta):
    i = torch.arange(n, device="cuda", dtype=torch.float64)
    return pos.double().unsqueeze(-1) * torch.exp(-math.log(theta) * i / n)


def _spin64(x, pos, theta):
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half].double(), x[..., half:].double())
    z = z * torch.polar(torch.ones((), device="cuda", dtype=torch.float64), _angle64(half, pos, theta))
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    L, H, D, G = c["layers"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    U, scale, th = L * H, c["dim"] ** -0.5, c["theta"]

    def block(x, offsets, b):
        a, e = offsets[b] * U, offsets[b + 1] * U
        return x[a:e].view(L, H, offsets[b + 1] - offsets[b], *x.shape[1:])

    if c["op"] == "shared":
        out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
        ck, cv = s["cache_k"].double(), s["cache_v"].double()
        for b in range(len(s["own_len"])):
            g, S = b // c["per_group"], s["own_len"][b]
            a, e = s["q_offsets"][b], s["q_offsets"][b + 1]
            P = s["prefix_len"][g]
            pos = P + S + torch.arange(e - a, device="cuda")
            bk, bv = block(ck, s["cache_offsets"], b), block(cv, s["cache_offsets"], b)
            bk[:, :, S:S + e - a] = _spin64(s["kq"][:, a:e], pos[:, None], th).transpose(1, 2)
            bv[:, :, S:S + e - a] = s["vq"][:, a:e].double().transpose(1, 2)
            for lay in range(L):
                # the appended keys enter as they are held, rounded to the cache's type
                k = torch.cat([block(s["prefix_k"], s["prefix_offsets"], g)[lay].double(),
                               bk[lay, :, :S + e - a].to(s["cache_k"].dtype).double()], 1)
                v = torch.cat([block(s["prefix_v"], s["prefix_offsets"], g)[lay].double(), bv[lay, :, :S + e - a]], 1)
                q = _spin64(s["q"][lay, a:e], pos[:, None], th).view(e - a, H, G, D)
                x = torch.einsum("thgd,hnd->thgn", q, k) * scale
                x = x.masked_fill(torch.arange(P + S + e - a, device="cuda") > pos[:, None, None, None], -math.inf)
                out[lay, a:e] = torch.einsum("thgn,hnd->thgd", torch.softmax(x, -1), v).reshape(e - a, H * G, D)
        return {"out": out, "cache_k": ck, "cache_v": cv}
    if c["op"] == "weights":
        w = s["weights"].double()
        for b in range(c["batch"]):
            P, a, e = s["prefix_len"][b], s["q_offsets"][b], s["q_offsets"][b + 1]
            n, pos = P + e - a, P + torch.arange(e - a, device="cuda")
            wb = block(w, s["cache_offsets"], b)
            for lay in range(L):
                q = _spin64(s["q"][lay, a:e], pos[:, None], th).view(e - a, H, G, D)
                x = torch.einsum("thgd,hnd->thgn", q, block(s["cache_k"], s["cache_offsets"], b)[lay, :, :n].double()) * scale
                x = x.masked_fill(torch.arange(n, device="cuda") > pos[:, None, None, None], -math.inf)
                p = torch.softmax(x, -1).sum((0, 2))
                wb[lay, :, :n] = p + (wb[lay, :, :n] if c["add"] else 0.0)
        return {"weights": w}
    dk, dv, dw = (s[k].double() for k in ("dst_k", "dst_v", "dst_weights"))
    for b in range(c["batch"]):
        n = s["kv_len"][b]
        keep = min(s["keep"][b], n)
        w = block(s["weights"], s["cache_offsets"], b)[:, :, :n]
        rest = w[:, :, c["first"]:n - c["recent"]].double()
        more = keep - c["first"] - c["recent"]
        mask = torch.ones((L, H, n), device="cuda", dtype=torch.bool)
        if keep < n:
            mask[:, :, c["first"]:n - c["recent"]] = False
            # distinct weights here: the more-th largest decides (equal ones go by place)
            top = torch.argsort(-rest, dim=-1, stable=True)[..., :more] + c["first"]
            mask.scatter_(2, top, True)
        idx = mask.nonzero()[:, 2].view(L, H, keep)
        i = torch.arange(keep, device="cuda").expand(L, H, keep)
        take = idx[..., None].expand(L, H, keep, D)
        k = block(s["cache_k"], s["cache_offsets"], b).gather(2, take)
        block(dk, s["dst_offsets"], b)[:, :, :keep] = _spin64(k, i - idx, th)
        block(dv, s["dst_offsets"], b)[:, :, :keep] = block(s["cache_v"], s["cache_offsets"], b).gather(2, take).double()
        block(dw, s["dst_offsets"], b)[:, :, :keep] = w.gather(2, idx).double()
    return {"kept": None, "dst_k": dk, "dst_v": dv, "dst_weights": dw}
