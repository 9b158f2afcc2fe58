"""Measured cases of the paged cache: appending keys and values to it, attention
over it (everything, or a window and the first rows), rows packed to 4 bits and
back, and attention over a cache whose older rows are packed.

Layouts are the library's: pages ``[n_pages, L, H_kv, page_rows, D]``; row r of
request b is row ``r % page_rows`` of page ``table[b][r // page_rows]``; a query
token's position is its row; queries are ``[L][T][H_q][D]``, not rotated; RoPE
pairs are (x_i, x_i+D/2).  A packed row is a scale per 32 dims and 4-bit codes.
"""
import math

import torch

own = False

# layers, query heads, kv heads, head dim, RoPE base of the served models
QWEN2_7B = dict(layers=28, q_heads=28, kv_heads=4, dim=128, theta=1e6, dtype="bf16")
QWEN3_8B = dict(layers=36, q_heads=32, kv_heads=8, dim=128, theta=1e6, dtype="bf16")
LLAMA31_8B = dict(layers=32, q_heads=32, kv_heads=8, dim=128, theta=5e5, dtype="bf16")
TINY = dict(layers=1, q_heads=4, kv_heads=2, dim=64, theta=1e4, dtype="fp32")

GROUP, BLOCK = 32, 32      # dims that share a scale; rows that are packed together


def listed():
    return [
        # the new token of every request of a serving batch
        dict(QWEN3_8B, name="append-step", op="append", batch=64, rows=1216, spread=300, q=1, page=64, turned=False),
        # one request's stitched prefix of five chunks goes to pages
        dict(QWEN2_7B, name="append-stitched", op="append", batch=1, rows=0, spread=0, q=2592, page=64, turned=True),
        # the small fp32 configuration: the query's 16 tokens
        dict(TINY, name="append-tiny", op="append", batch=1, rows=193, spread=0, q=16, page=16, turned=False),
        # one request's prefix is packed, and restored
        dict(QWEN2_7B, name="pack-one", op="pack", batch=1, rows=2592, spread=0, begin=0, page=64),
        # the pages that a serving batch filled lately
        dict(QWEN3_8B, name="pack-batch", op="pack", batch=32, rows=1216, spread=300, begin=1088, page=64),
        # a decode step of four users over their own caches
        dict(QWEN2_7B, name="paged-decode", op="paged", batch=4, rows=2655, spread=63, q=1, page=64, window=0, first=0),
        # long sessions, a window of 4,096 tokens and the first four
        dict(LLAMA31_8B, name="paged-window", op="paged", batch=8, rows=6000, spread=1500, q=1, page=16, window=4096, first=4),
        # a prompt without a stitched prefix, window of 1,024
        dict(LLAMA31_8B, name="paged-prompt", op="paged", batch=1, rows=0, spread=0, q=4096, page=64, window=1024, first=64),
        # the small fp32 configuration: 16 tokens behind 193
        dict(TINY, name="paged-tiny", op="paged", batch=1, rows=193, spread=0, q=16, page=16, window=0, first=0),
        # a serving batch's decode step, all but the last rows in 4 bits
        dict(QWEN3_8B, name="packed-decode", op="packed", batch=16, rows=1216, spread=300, q=1, page=64, window=0, first=0, tail=64),
        # a 32k-token document cache in 4 bits
        dict(LLAMA31_8B, name="packed-32k", op="packed", batch=1, rows=33280, spread=0, q=1, page=64, window=0, first=0, tail=96),
        # eight questions of 64 tokens over packed prefixes
        dict(QWEN2_7B, name="packed-query", op="packed", batch=8, rows=2592, spread=95, q=64, page=32, window=0, first=0, tail=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "pack", "paged", "packed", "paged", "packed"))
    models = (QWEN2_7B, QWEN3_8B, LLAMA31_8B, QWEN2_7B, QWEN3_8B, LLAMA31_8B)
    m = dict(rng.choice(models if op in ("pack", "packed") else models + (TINY,)))
    m["layers"] = rng.randint(1, m["layers"])
    tiny = m["dim"] == 64
    if tiny:
        m["dtype"] = rng.choice(("fp32", "bf16"))
    units = m["layers"] * m["kv_heads"]
    page = rng.choice((32, 64, 128, 96)) if op in ("pack", "packed") else rng.choice((16, 32, 64, 128, 48, 20))
    batch = _log(rng, 1, 3 if tiny else 24)
    top = 2000 if tiny else 24000
    # rows of all requests, within the largest listed cache
    rows = _log(rng, 40, min(top, max(64, 256 * 33280 // (units * batch))))
    spread = rng.randint(0, rows // 2)
    if op == "append":
        q = rng.choice((1, 1, _log(rng, 2, max(3, min(2000, 112 * 2592 // (units * batch))))))
        return dict(m, op=op, batch=batch, rows=rows, spread=spread, q=q, page=page, turned=rng.choice((True, False)))
    if op == "pack":
        rows = max(64, min(rows // 3, 8192))
        return dict(m, op=op, batch=batch, rows=rows, spread=min(spread, rows - 33), begin=rng.choice((0, rows // 4)), page=page)
    q = rng.choice((1, 1, 1, rng.randint(2, 12), rng.randint(13, 200)))
    window = rng.choice((0, 0, _log(rng, 8, max(9, rows))))
    if tiny or page % 16:    # few query rows on the CUDA cores
        rows, q, m["layers"], batch = min(rows, 2000), min(q, 24), min(m["layers"], 4), min(batch, 4)
        spread = min(spread, rows // 2)
    while batch * q * rows * units > 8 * 64 * 2592 * 112:
        q = max(1, q // 2)
        rows = max(40, rows // 2)
        spread = min(spread, rows // 2)
    c = dict(m, op=op, batch=batch, rows=rows, spread=spread, q=q, page=page, window=window,
             first=rng.randint(0, 80) if window else 0)
    if op == "packed":
        c["tail"] = rng.randint(0, 160)
    return c


# ---- sizes of a case ----
def _ragged(base, spread, n):
    """n lengths in [base - spread, base], from the case alone."""
    return [base - (i * 7919) % (spread + 1) for i in range(n)]


def _starts(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _sizes(c):
    """Rows before the call, query tokens, rows packed, of each request."""
    before = _ragged(c["rows"], c["spread"], c["batch"])
    if c["op"] == "pack":
        return before, None, None
    q = _ragged(c["q"], min(c["spread"], c["q"] // 3), c["batch"])
    packed = [max(0, p + t - c["tail"]) // BLOCK * BLOCK for p, t in zip(before, q)] if c["op"] == "packed" else None
    return before, q, packed


def _pack_range(c, n):
    """Rows of a request of n rows that a pack call takes: whole blocks."""
    return min(c["begin"], n) // BLOCK * BLOCK, n // BLOCK * BLOCK


def _pairs(p, t, window, first):
    """Keys that the tokens at positions p .. p + t - 1 see, in all."""
    if not window:
        return t * p + t * (t + 1) // 2
    return sum(min(window, x + 1) + min(first, max(0, x - window + 1)) for x in range(p, p + t))


def _seen(p, t, window, first):
    """Rows that some of these tokens see: the first ones [0, a) and [lo, p + t)."""
    lo = max(0, p - window + 1) if window else 0
    return min(first, lo), lo


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    D, L, Hq, H = c["dim"], c["layers"], c["q_heads"], c["kv_heads"]
    row = 2 * L * H * D * e                                # one token's keys and values
    thin = 2 * L * H * (D // 2 + D // GROUP * 2)           # packed
    before, q, packed = _sizes(c)
    if c["op"] == "append":
        return {"bytes": 2 * row * sum(q), "flops": 0 if c["turned"] else 3 * D * L * H * sum(q)}
    if c["op"] == "pack":
        n = sum(b - a for a, b in (_pack_range(c, x) for x in before))
        return {"bytes": 2 * (row + thin) * n, "flops": 2 * 3 * 2 * D * L * H * n}
    rows = few = pairs = 0
    for i, (p, t) in enumerate(zip(before, q)):
        a, lo = _seen(p, t, c["window"], c["first"])
        n, body = p + t, packed[i] if packed else 0
        few += min(a, body) + max(0, body - lo)
        rows += a - min(a, body) + n - max(lo, body)
        pairs += _pairs(p, t, c["window"], c["first"])
    return {"bytes": row * rows + thin * few + 2 * sum(q) * L * Hq * D * e, "flops": 4 * D * Hq * L * pairs}


# ---- inputs ----
def _pool(c):
    """The handle a program keeps: a pool of this layout (its chunks are not read here)."""
    from rag_precomputed_kv_gb300 import kvr
    k = torch.zeros((1, c["layers"], c["kv_heads"], 8, c["dim"]), device="cuda", dtype=_dtype(c))
    return kvr.Pool(k, torch.zeros_like(k), c["q_heads"], c["theta"])


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _table(c, rows, seed):
    """A page table of requests of so many rows, in a shuffled pool with three spare pages."""
    need = [-(-r // c["page"]) for r in rows]
    ids = torch.randperm(sum(need) + 3, generator=torch.Generator().manual_seed(seed), dtype=torch.int64).to(torch.int32)
    table = torch.full((len(rows), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + 3


def prepare(case, seed):
    c, dt = case, _dtype(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    D, L, Hq, H, R = c["dim"], c["layers"], c["q_heads"], c["kv_heads"], c["page"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    before, q, packed = _sizes(c)
    total = [p + t for p, t in zip(before, q)] if q else before
    table, n_pages = _table(c, total, seed)
    s = {"case": c, "table": table, "k": randn(n_pages, L, H, R, D), "v": randn(n_pages, L, H, R, D)}
    if own:
        from rag_precomputed_kv_gb300 import kvr
        s["pool"] = _pool(c)
        s["pages"] = kvr.Pages(s["k"], s["v"])
    if c["op"] == "append":
        T = sum(q)
        s.update(start=before, q_offsets=_starts(q))
        if c["turned"]:    # a stitched cache, [L][H][rows][D], seen token by token
            s.update(new_k=randn(L, H, T, D).transpose(1, 2), new_v=randn(L, H, T, D).transpose(1, 2))
        else:
            s.update(new_k=randn(L, T, H, D), new_v=randn(L, T, H, D))
    elif c["op"] == "pack":
        spans = [_pack_range(c, n) for n in before]
        s.update(begin=[a for a, _ in spans], end=[b for _, b in spans], to_k=torch.zeros_like(s["k"]), to_v=torch.zeros_like(s["v"]))
        if own:
            s["to"] = kvr.Pages(s["to_k"], s["to_v"])
            s["packed"] = s["pool"].packed_pages(n_pages, R)
    else:
        T = sum(q)
        s.update(kv_len=total, q_offsets=_starts(q), q=randn(L, T, Hq, D), out=torch.zeros((L, T, Hq, D), device="cuda", dtype=dt))
        if c["op"] == "packed":
            s["packed_len"] = packed
            if own:
                s["packed"] = s["pool"].packed_pages(n_pages, R)
                s["pool"].page_pack(s["pages"], table, s["packed"], table, [0] * len(packed), packed)
            else:    # every row's codes and scales; those behind packed_len are not read
                for x in ("k", "v"):
                    codes, scales = zip(*(_codes(y) for y in s[x].split(64)))
                    s[x + "_codes"], s[x + "_scales"] = torch.cat(codes), torch.cat(scales)
    return s


# ---- one pass ----
def run(state):
    s, c = state, state["case"]
    if c["op"] == "append":
        if own:
            s["pool"].page_append(s["pages"], s["table"], s["start"], s["q_offsets"], s["new_k"], s["new_v"], turned=c["turned"])
        else:
            _plain_append(s, c)
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "pack":
        if own:
            s["pool"].page_pack(s["pages"], s["table"], s["packed"], s["table"], s["begin"], s["end"])
            s["pool"].page_unpack(s["packed"], s["table"], s["to"], s["table"], s["begin"], s["end"])
        else:
            _plain_pack(s, c)
        return {"k": s["to_k"], "v": s["to_v"]}
    if own and c["op"] == "packed":
        s["pool"].page_attention(s["pages"], s["table"], s["kv_len"], s["q_offsets"], s["q"], s["out"], window=c["window"],
                                 n_first=c["first"], packed=s["packed"], packed_table=s["table"], packed_len=s["packed_len"])
    elif own:
        s["pool"].page_attention(s["pages"], s["table"], s["kv_len"], s["q_offsets"], s["q"], s["out"], window=c["window"],
                                 n_first=c["first"])
    else:
        _plain_attention(s, c)
    return {"out": s["out"]}


# ---- the plain forms ----
def _turn(x, pos, theta):
    """x [..., D] in fp32 turned by pos [...]; the angles in 64 bits."""
    h = x.shape[-1] // 2
    w = theta ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    a = pos[..., None].double() * w
    co, si = torch.cos(a).float(), torch.sin(a).float()
    lo, hi = x[..., :h], x[..., h:]
    return torch.cat([lo * co - hi * si, lo * si + hi * co], -1)


def _place(s, c, b, rows):
    """Pages, and rows in them, of these rows of request b."""
    return s["table"].to("cuda", torch.int64)[b, rows // c["page"]], rows % c["page"]


def _codes(x):
    """Codes (-7 .. 7) and bf16 scales of rows of bf16 values, 32 dims to a scale."""
    y = x.float().unflatten(-1, (-1, GROUP))
    scale = (y.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16)
    codes = torch.where(scale > 0, torch.round(y / scale.float()), 0.0).clamp(-7, 7).to(torch.int8)
    return codes.flatten(-2), scale.squeeze(-1)


def _values(codes, scales):
    return (codes.float().unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _plain_append(s, c):
    at = [torch.arange(p, p + b - a, device="cuda") for p, a, b in zip(s["start"], s["q_offsets"], s["q_offsets"][1:])]
    page, row = (torch.cat(x) for x in zip(*(_place(s, c, b, r) for b, r in enumerate(at))))
    k = s["new_k"]
    if not c["turned"]:
        k = _turn(k.float(), torch.cat(at)[:, None], c["theta"]).to(k.dtype)
    s["k"][page, :, :, row] = k.transpose(0, 1)
    s["v"][page, :, :, row] = s["new_v"].transpose(0, 1)


def _plain_pack(s, c):
    for b, (begin, end) in enumerate(zip(s["begin"], s["end"])):
        page, row = _place(s, c, b, torch.arange(begin, end, device="cuda"))
        for x in ("k", "v"):
            s["to_" + x][page, :, :, row] = _values(*_codes(s[x][page, :, :, row])).to(s[x].dtype)


def _plain_attention(s, c):
    L, H, D, G = c["layers"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    W, S, scale, step = c["window"], c["first"], 1.0 / math.sqrt(c["dim"]), 512
    for b, n in enumerate(s["kv_len"]):
        t0, t1 = s["q_offsets"][b], s["q_offsets"][b + 1]
        for a in range(t0, t1, step):
            e = min(t1, a + step)
            pos = torch.arange(n - t1 + a, n - t1 + e, device="cuda")
            few, lo = _seen(n - t1 + a, e - a, W, S)
            rows = torch.cat([torch.arange(few, device="cuda"), torch.arange(lo, n - t1 + e, device="cuda")])
            page, row = _place(s, c, b, rows)
            sees = rows <= pos[:, None]
            if W:
                sees &= (rows > pos[:, None] - W) | (rows < S)
            # as many layers at a time as keep the scores within a few GB
            per = max(1, min(L, 2 ** 29 // (H * G * (e - a) * len(rows)), 2 ** 29 // (H * D * len(rows))))
            for l0 in range(0, L, per):
                l1 = min(L, l0 + per)

                def held(x):    # [m, layers, H, D] -> [layers, H, m, D]
                    y = s[x][:, l0:l1][page, :, :, row].float()
                    if c["op"] == "packed":
                        z = _values(s[x + "_codes"][:, l0:l1][page, :, :, row], s[x + "_scales"][:, l0:l1][page, :, :, row])
                        y = torch.where((rows < s["packed_len"][b])[:, None, None, None], z, y)
                    return y.permute(1, 2, 0, 3)

                x = _turn(s["q"][l0:l1, a:e].float(), pos[:, None], c["theta"])
                x = x.view(l1 - l0, e - a, H, G, D).permute(0, 2, 1, 3, 4).reshape(l1 - l0, H, -1, D)
                p = x @ held("k").transpose(-1, -2) * scale
                p.masked_fill_(~sees.repeat_interleave(G, 0), -math.inf)
                p = torch.exp(p.sub_(p.amax(-1, keepdim=True)))
                o = (p @ held("v")).div_(p.sum(-1, keepdim=True))
                s["out"][l0:l1, a:e] = o.view(l1 - l0, H, e - a, G, D).transpose(1, 2).reshape(l1 - l0, e - a, H * G, D).to(s["out"].dtype)


# ---- the definitions in 64 bits, request by request ----
def _spin64(x, pos, theta):
    half = x.shape[-1] // 2
    turn = pos.double().unsqueeze(-1) * torch.exp(-math.log(theta) * torch.arange(half, device="cuda", dtype=torch.float64) / half)
    z = torch.complex(x[..., :half].double(), x[..., half:].double())
    z = z * torch.polar(torch.ones((), device="cuda", dtype=torch.float64), turn)
    return torch.cat([z.real, z.imag], -1)


def _thin64(x):
    """What packed rows stand for: multiples of a bf16 scale, in 64 bits."""
    parts = []
    for y in x.double().split(GROUP, -1):
        unit = (y.abs().max(-1, keepdim=True).values / 7.0).to(torch.bfloat16).double()
        parts.append(torch.where(unit > 0, torch.round(y / torch.where(unit > 0, unit, 1.0)), 0.0).clamp(-7, 7) * unit)
    return torch.cat(parts, -1)


def _rows64(s, c, x, b, n, lay):
    """Rows 0 .. n - 1 of request b in a layer of pages x: [H, n, D], as they are held."""
    ids = s["table"][b, :-(-n // c["page"])].tolist()
    return torch.cat([x[i, lay] for i in ids], 1)[:, :n]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    L, H, D, G, R = c["layers"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"], c["page"]
    if c["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        for b, p in enumerate(s["start"]):
            for t in range(s["q_offsets"][b], s["q_offsets"][b + 1]):
                r = p + t - s["q_offsets"][b]
                i = int(s["table"][b, r // R])
                new = s["new_k"][:, t].double()
                k[i, :, :, r % R] = new if c["turned"] else _spin64(new, torch.full((1, 1), r, device="cuda"), c["theta"])
                v[i, :, :, r % R] = s["new_v"][:, t].double()
        return {"k": k, "v": v}
    if c["op"] == "pack":
        k, v = torch.zeros_like(s["k"], dtype=torch.float64), torch.zeros_like(s["v"], dtype=torch.float64)
        for b, (begin, end) in enumerate(zip(s["begin"], s["end"])):
            for r in range(begin, end, BLOCK):
                i, a = int(s["table"][b, r // R]), r % R
                k[i, :, :, a:a + BLOCK] = _thin64(s["k"][i, :, :, a:a + BLOCK])
                v[i, :, :, a:a + BLOCK] = _thin64(s["v"][i, :, :, a:a + BLOCK])
        return {"k": k, "v": v}
    out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    for b, n in enumerate(s["kv_len"]):
        t0, t1 = s["q_offsets"][b], s["q_offsets"][b + 1]
        body = s["packed_len"][b] if c["op"] == "packed" else 0
        for lay in range(L):
            k, v = (_rows64(s, c, s[x], b, n, lay).double() for x in ("k", "v"))
            if body:
                k[:, :body], v[:, :body] = _thin64(k[:, :body]), _thin64(v[:, :body])
            for a in range(t0, t1, 256):
                e = min(t1, a + 256)
                pos = n - t1 + torch.arange(a, e, device="cuda")
                j = torch.arange(n, device="cuda")
                hide = j > pos[:, None]
                if c["window"]:
                    hide = hide | ((pos[:, None] - j >= c["window"]) & (j >= c["first"]))
                used = (~hide).any(0).nonzero().squeeze(1)         # keys that no token of these sees are left out
                q = _spin64(s["q"][lay, a:e], pos[:, None], c["theta"]).view(e - a, H, G, D)
                x = torch.einsum("thgd,hnd->thgn", q, k[:, used]) * D ** -0.5
                x = x.masked_fill(hide[:, used][:, None, None], -math.inf)
                out[lay, a:e] = torch.einsum("thgn,hnd->thgd", torch.softmax(x, -1), v[:, used]).reshape(e - a, H * G, D)
    return {"out": out}
