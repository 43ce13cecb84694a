"""The operators of a serving step around the GEMMs: rotary positions with per-head norms, the
same written into a paged key/value cache, and attention that reads such a cache (its batch may
share a long prefix). ``run`` computes them in plain torch operations, or through the library
when ``own`` is true; ``exact`` computes them again in 64 bits.

A batch is ragged: sequence s has the tokens q_start[s] .. q_start[s + 1] - 1 of the flat token
dimension and, once they are appended, kv_lens[s] keys of its own, held in the pages
page_table[s][0], page_table[s][1], ... of the cache. Keys of a shared prefix come before them.
Token i of n new ones stands at position prefix + kv_len - n + i and sees the keys up to there.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda:0"
EPS = 1e-6
TURN = 2.0 * math.pi
_GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------------- the cases

def _rope(name, **kw):
    d = dict(name=name, op="qk_rope", dtype="float16", tokens=1, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, interleaved=False, norm=True, base=10000.0, factor=1.0, rope_scale=1.0,
             first=0, heads_out=False)
    d.update(kw)
    return d


def _append(name, **kw):
    d = dict(name=name, op="kv_append", dtype="float16", seqs=1, q_min=1, q_max=1, ctx_min=0, ctx_max=0,
             q_heads=32, kv_heads=8, head_dim=128, page_size=16, by_rows=False, prefix_pages=0,
             rotary_dim=128, interleaved=False, norm=True, base=10000.0, factor=1.0, rope_scale=1.0)
    d.update(kw)
    return d


def _attend(name, **kw):
    d = dict(name=name, op="paged_attention", dtype="float16", seqs=1, q_min=1, q_max=1, ctx_min=0, ctx_max=0,
             q_heads=32, kv_heads=8, head_dim=128, page_size=16, by_rows=False, prefix_pages=0)
    d.update(kw)
    return d


def listed():
    return [
        # one new token of one user: the latency of a call
        _rope("rope_token", first=4095),
        # a prompt of the MLP benchmark's 8200 tokens, laid out head by head for the contiguous attention
        _rope("rope_prompt_by_head", tokens=8200, kv_heads=32, norm=False, heads_out=True),
        # a decoding step of 64 users far into their texts, part of each head rotated, positions interpolated
        _append("append_step", dtype="bfloat16", seqs=64, ctx_min=3, ctx_max=100000, rotary_dim=64, interleaved=True,
                factor=4.0, rope_scale=1.1),
        # five prompts of ragged lengths written into a token-major cache
        _append("append_prompts", seqs=5, q_min=100, q_max=4001, page_size=64, by_rows=True),
        # one new token of one user with a short text
        _attend("attend_token", ctx_min=776, ctx_max=776),
        # a decoding step of 64 users whose texts differ much in length
        _attend("attend_step", dtype="bfloat16", seqs=64, ctx_min=15, ctx_max=8191, page_size=64),
        # two very long texts: the split over the keys
        _attend("attend_step_far", seqs=2, ctx_min=131000, ctx_max=131071, page_size=256),
        # many users with up to three drafted tokens each, one key head per query head, heads of 64
        _attend("attend_drafts_d64", seqs=200, q_max=3, ctx_max=2000, q_heads=16, kv_heads=16, head_dim=64, by_rows=True),
        # three fresh prompts: compute bound
        _attend("attend_prompts", seqs=3, q_min=129, q_max=4096, kv_heads=32, page_size=128),
        # a mixed step: pieces of long prompts beside single tokens
        _attend("attend_mixed", dtype="bfloat16", seqs=9, q_max=512, ctx_min=1000, ctx_max=16000, page_size=32),
        # 48 users with the same 16480-token prefix and short texts of their own
        _attend("shared_step", seqs=48, ctx_max=700, page_size=32, prefix_pages=515),
        # a few users with drafted tokens behind a medium prefix, heads of 64
        _attend("shared_drafts_d64", dtype="bfloat16", seqs=7, q_max=5, ctx_max=300, q_heads=24, kv_heads=4, head_dim=64,
                prefix_pages=127),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_rope", "kv_append", "paged_attention", "paged_attention"])
    c = dict(op=op, dtype=rng.choice(["float16", "bfloat16"]))
    head_dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    c.update(head_dim=head_dim, kv_heads=kv_heads, q_heads=kv_heads * group)
    if op != "paged_attention":
        c.update(rotary_dim=16 * rng.randint(1, head_dim // 16), interleaved=rng.random() < 0.5, norm=rng.random() < 0.5,
                 base=rng.choice([10000.0, 500000.0, 1000000.0]), factor=rng.choice([1.0, 1.0, 8.0]),
                 rope_scale=rng.choice([1.0, 1.0, 1.2]))
    if op == "qk_rope":
        c.update(tokens=_log(rng, 1, 8200), first=_log(rng, 1, 1000000), heads_out=rng.random() < 0.5)
        return c
    c.update(page_size=rng.choice([16, 32, 64, 128, 256]), by_rows=rng.random() < 0.5,
             prefix_pages=0 if rng.random() < 0.6 else _log(rng, 1, 100))
    if rng.random() < 0.6:   # a decoding step
        seqs, q_max = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 5])
        ctx_max = _log(rng, 16, min(131072, 200000000 // (seqs * kv_heads * head_dim) + 64))
    else:                    # prompts or pieces of them
        seqs, q_max = _log(rng, 1, 16), _log(rng, 8, 4096)
        q_max = min(q_max, 12000 // seqs)
        ctx_max = rng.choice([0, _log(rng, 16, 12000 // seqs + 32)])
        if op == "paged_attention":   # the plain form holds all scores
            total = ctx_max + q_max + c["prefix_pages"] * c["page_size"]
            q_max = max(1, min(q_max, int(6.4e10 / (seqs * c["q_heads"] * total * head_dim))))
    q_min = rng.randint(1, q_max)
    c.update(seqs=seqs, q_min=q_min, q_max=q_max, ctx_min=rng.randint(0, ctx_max), ctx_max=ctx_max)
    return c


def _spread(n, lo, hi, phase):
    """n whole numbers from lo to hi, spread over their logarithm, in a scrambled order."""
    if n == 1:
        return [hi]
    at = [((i * _GOLDEN + phase) % 1.0) for i in range(n)]
    order = sorted(range(n), key=lambda i: at[i])
    rank = [0] * n
    for k, i in enumerate(order):
        rank[i] = k
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (r / (n - 1)))) - 1 for r in rank]


def _lengths(c):
    """New tokens and own keys (the new ones among them) of each sequence."""
    n_q = _spread(c["seqs"], c["q_min"], c["q_max"], 0.3)
    ctx = _spread(c["seqs"], c["ctx_min"], c["ctx_max"], 0.0)
    return n_q, [a + b for a, b in zip(n_q, ctx)]


# ---------------------------------------------------------------------------------- the inputs

def _frequencies(c):
    """Radians a position turns each pair of a head, in 64 bits."""
    half = c["rotary_dim"] // 2
    return c["base"] ** (-np.arange(half, dtype=np.float64) / half) / c["factor"]


def _table(freq):
    """The library's form of the frequencies: turns a position in units of 2^-64, as 64-bit words."""
    return np.round(freq / TURN * 2.0 ** 64).astype(np.uint64).view(np.int64)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = getattr(torch, c["dtype"])
    hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32) * scale).to(dt)

    s = dict(case=dict(c))
    if c["op"] != "paged_attention":
        freq = _frequencies(c)
        s["freq"] = torch.from_numpy(freq).to(DEVICE)
        s["table"] = torch.from_numpy(_table(freq)).to(DEVICE)
        s["q_norm"] = (1 + 0.2 * normal(d).float()).to(dt) if c["norm"] else None
        s["k_norm"] = (1 + 0.2 * normal(d).float()).to(dt) if c["norm"] else None
    if c["op"] == "qk_rope":
        t = c["tokens"]
        qkv = normal(t, (hq + 2 * hk) * d)   # the packed projection of a layer
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d : (hq + hk) * d].unflatten(1, (hk, d))
        s["positions"] = torch.arange(c["first"], c["first"] + t, device=DEVICE, dtype=torch.int32)
        return s
    n_q, kv = _lengths(c)
    ps, n = c["page_size"], c["seqs"]
    tokens = sum(n_q)
    need = [-(-x // ps) for x in kv]
    width = max(need)
    pages = sum(need) + c["prefix_pages"] + 2
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32).cpu()
    table = torch.zeros(n, width, dtype=torch.int32)
    at = c["prefix_pages"]
    for i, w in enumerate(need):
        table[i, :w] = order[at : at + w]
        at += w
    s["page_table"] = table.to(DEVICE)
    s["prefix_pages"] = order[: c["prefix_pages"]].to(DEVICE) if c["prefix_pages"] else None
    s["q_start"] = torch.tensor(np.cumsum([0] + n_q), dtype=torch.int32, device=DEVICE)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEVICE)
    s["max_q"], s["max_kv"], s["tokens"] = max(n_q), max(kv), tokens
    shape = (pages, ps, hk, d) if c["by_rows"] else (pages, hk, ps, d)
    cache = [normal(*shape) for _ in range(2)]
    s["k_cache"], s["v_cache"] = [x.transpose(1, 2) if c["by_rows"] else x for x in cache]   # [page, head, row, dim]
    qkv = normal(tokens, (hq + 2 * hk) * d)
    s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
    if c["op"] == "kv_append":
        s["k"] = qkv[:, hq * d : (hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d :].unflatten(1, (hk, d))
    else:
        s["q"] = normal(tokens, hq, d)
    return s


# ------------------------------------------------------------------------------ the plain form

def _norm_rotate(x, weight, cos, sin, c):
    """x [tokens, heads, dim]: the norm of each head, then the rotation of its first rotary_dim entries."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    rd = c["rotary_dim"]
    r, rest = y[..., :rd], y[..., rd:]
    cos, sin = cos[:, None], sin[:, None]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., : rd // 2], r[..., rd // 2 :]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1).to(x.dtype)


def _angles(positions, s):
    a = positions.double()[:, None] * s["freq"]
    scale = s["case"]["rope_scale"]
    return (a.cos() * scale).float(), (a.sin() * scale).float()


def _token_places(s):
    """Of each token: its sequence and its place among that sequence's own keys."""
    q_start = s["q_start"].long()
    t = torch.arange(s["tokens"], device=DEVICE)
    seq = torch.searchsorted(q_start, t, right=True) - 1
    n_q = q_start[1:] - q_start[:-1]
    return seq, s["kv_lens"].long()[seq] - n_q[seq] + t - q_start[seq]


def _plain_qk_rope(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], s)
    q = _norm_rotate(s["q"], s["q_norm"], cos, sin, c)
    k = _norm_rotate(s["k"], s["k_norm"], cos, sin, c)
    return {"q": q.transpose(0, 1).contiguous() if c["heads_out"] else q,
            "k": k.transpose(0, 1).contiguous() if c["heads_out"] else k}


def _plain_kv_append(s):
    c = s["case"]
    seq, place = _token_places(s)
    cos, sin = _angles(place + c["prefix_pages"] * c["page_size"], s)
    page = s["page_table"].long()[seq, place // c["page_size"]]
    row = place % c["page_size"]
    s["k_cache"][page, :, row] = _norm_rotate(s["k"], s["k_norm"], cos, sin, c)
    s["v_cache"][page, :, row] = s["v"]
    return {"q": _norm_rotate(s["q"], s["q_norm"], cos, sin, c), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_paged_attention(s):
    c = s["case"]
    hq, hk, d, ps, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["page_size"], c["seqs"]
    g, mq, tokens = hq // hk, s["max_q"], s["tokens"]
    prefix = c["prefix_pages"] * ps
    q_start, kv_lens = s["q_start"].long(), s["kv_lens"].long()
    n_q = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=DEVICE)
    token = (q_start[:-1, None] + i).clamp(max=tokens - 1)                     # [n, mq]
    place = kv_lens[:, None] - n_q[:, None] + i                                # own keys up to here are seen
    q = s["q"].float()[token].view(n, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * mq, d)

    def keys(cache, pages):   # [..., pages] -> [..., heads, keys, dim]
        x = cache[pages.long()].float().transpose(-4, -3)
        return x.flatten(-3, -2)

    k, v = keys(s["k_cache"], s["page_table"]), keys(s["v_cache"], s["page_table"])
    at = torch.arange(k.shape[2], device=DEVICE)
    v = v * (at < kv_lens[:, None])[:, None, :, None]
    score = (q @ k.transpose(-1, -2)).view(n, hk, g, mq, -1) * (1.0 / math.sqrt(d))
    score = score.masked_fill(at > place[:, None, None, :, None], -math.inf)
    if prefix:
        kp, vp = keys(s["k_cache"], s["prefix_pages"]), keys(s["v_cache"], s["prefix_pages"])
        qp = q.transpose(0, 1).reshape(hk, n * g * mq, d)
        before = (qp @ kp.transpose(-1, -2)).view(hk, n, g, mq, prefix).transpose(0, 1) * (1.0 / math.sqrt(d))
        score = torch.cat((before, score), -1)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = p[..., prefix:].reshape(n, hk, g * mq, -1) @ v
    if prefix:
        before = p[..., :prefix].transpose(0, 1).reshape(hk, n * g * mq, prefix) @ vp
        o = o + before.view(hk, n, g * mq, d).transpose(0, 1)
    o = (o.view(n, hk, g, mq, d) / total).permute(0, 3, 1, 2, 4).reshape(n, mq, hq, d)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(n, mq, hq)
    # back to the flat tokens: the padding goes to a row behind the last
    to = torch.where(i < n_q[:, None], token, tokens)
    out = torch.empty(tokens + 1, hq, d, device=DEVICE, dtype=s["q"].dtype)
    out[to] = o.to(out.dtype)
    out_lse = torch.empty(tokens + 1, hq, device=DEVICE, dtype=torch.float32)
    out_lse[to] = lse
    return {"out": out[:tokens], "lse": out_lse[:tokens]}


# ------------------------------------------------------------------------- the library's calls

_context = None


def _library():
    global _context
    import tensor_core_gemm_tcgen05_gb300 as g
    if _context is None:
        _context = g.Context(0)
    return g, _context


def _own_qk_rope(s):
    g, ctx = _library()
    c = s["case"]
    q_out = k_out = None
    if c["heads_out"]:
        q_out = torch.empty(c["q_heads"], c["tokens"], c["head_dim"], dtype=s["q"].dtype, device=DEVICE).transpose(0, 1)
        k_out = torch.empty(c["kv_heads"], c["tokens"], c["head_dim"], dtype=s["q"].dtype, device=DEVICE).transpose(0, 1)
    q, k = g.qk_rope(ctx, s["q"], s["k"], s["positions"], s["table"], interleaved=c["interleaved"],
                     rope_scale=c["rope_scale"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, q_out=q_out, k_out=k_out)
    return {"q": q.transpose(0, 1), "k": k.transpose(0, 1)} if c["heads_out"] else {"q": q, "k": k}


def _own_kv_append(s):
    g, ctx = _library()
    c = s["case"]
    q = g.kv_append(ctx, s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_lens"], s["page_table"],
                    s["table"], prefix_len=c["prefix_pages"] * c["page_size"], interleaved=c["interleaved"],
                    rope_scale=c["rope_scale"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_paged_attention(s):
    g, ctx = _library()
    lse = torch.empty(s["tokens"], s["case"]["q_heads"], dtype=torch.float32, device=DEVICE)
    out = g.paged_attention(ctx, s["q"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_lens"], s["page_table"],
                            max_q=s["max_q"], prefix_pages=s["prefix_pages"], lse=lse)
    return {"out": out, "lse": lse}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"qk_rope": _own_qk_rope, "kv_append": _own_kv_append, "paged_attention": _own_paged_attention}[op](state)
    return {"qk_rope": _plain_qk_rope, "kv_append": _plain_kv_append, "paged_attention": _plain_paged_attention}[op](state)


# ------------------------------------------------------------------------- what a pass has to do

def work(case):
    c = case
    hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "qk_rope":
        t = c["tokens"]
        values = t * (hq + hk) * d
        return {"bytes": 4 * values + 4 * t, "flops": values * (7 if c["norm"] else 3)}
    n_q, kv = _lengths(c)
    t, ps = sum(n_q), c["page_size"]
    prefix = c["prefix_pages"] * ps
    if c["op"] == "kv_append":
        values = t * (hq + 2 * hk) * d
        return {"bytes": 4 * values + 8 * c["seqs"], "flops": t * (hq + hk) * d * (7 if c["norm"] else 3)}
    seen = sum(n * (prefix + k) - n * (n - 1) // 2 for n, k in zip(n_q, kv))
    keys = prefix + sum(kv)
    tables = 4 * (2 * c["seqs"] + c["prefix_pages"] + sum(-(-k // ps) for k in kv))
    return {"bytes": 4 * t * hq * d + 4 * t * hq + 4 * keys * hk * d + tables, "flops": 4 * d * hq * seen}


# --------------------------------------------------------------------------- in 64 bits, apart

def _exact_head(x, weight, position, freq, c):
    """One tensor [tokens, heads, dim] by the definition, with complex numbers for the rotation."""
    y = x.double()
    if weight is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * weight.double()
    half = c["rotary_dim"] // 2
    turn = torch.polar(torch.full_like(freq, c["rope_scale"])[None] + 0 * position.double()[:, None], position.double()[:, None] * freq)
    first = torch.arange(half, device=DEVICE)
    one, two = (2 * first, 2 * first + 1) if c["interleaved"] else (first, first + half)
    z = torch.complex(y[..., one], y[..., two]) * turn[:, None]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    hq, hk, d, g = c["q_heads"], c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    if c["op"] == "qk_rope":
        out = {}
        for name in ("q", "k"):
            y = _exact_head(s[name], s[name + "_norm"], s["positions"], s["freq"], c)
            out[name] = y.transpose(0, 1).contiguous() if c["heads_out"] else y
        return out
    n_q, kv = _lengths(c)
    ps, prefix = c["page_size"], c["prefix_pages"] * c["page_size"]
    starts = np.cumsum([0] + n_q)
    if c["op"] == "kv_append":
        k_cache, v_cache, q = s["k_cache"].double(), s["v_cache"].double(), s["q"].double()
        for i in range(c["seqs"]):
            a, b = int(starts[i]), int(starts[i + 1])
            place = torch.arange(kv[i] - n_q[i], kv[i], device=DEVICE)
            page, row = s["page_table"][i].long()[place // ps], place % ps
            q[a:b] = _exact_head(s["q"][a:b], s["q_norm"], place + prefix, s["freq"], c)
            k_cache[page, :, row] = _exact_head(s["k"][a:b], s["k_norm"], place + prefix, s["freq"], c)
            v_cache[page, :, row] = s["v"][a:b].double()
        return {"q": q, "k_cache": k_cache, "v_cache": v_cache}
    if work(c)["flops"] > 4e12:
        return None
    out = torch.empty(s["tokens"], hq, d, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["tokens"], hq, dtype=torch.float64, device=DEVICE)
    for i in range(c["seqs"]):
        a, b = int(starts[i]), int(starts[i + 1])
        pages = s["page_table"][i, : -(-kv[i] // ps)]
        if prefix:
            pages = torch.cat((s["prefix_pages"], pages))
        last = prefix + kv[i] - n_q[i] + torch.arange(n_q[i], device=DEVICE)
        for h in range(hk):
            k = s["k_cache"][pages.long(), h].double().flatten(0, 1)[: prefix + kv[i]]
            v = s["v_cache"][pages.long(), h].double().flatten(0, 1)[: prefix + kv[i]]
            hidden = torch.arange(prefix + kv[i], device=DEVICE) > last[:, None]
            for j in range(h * g, (h + 1) * g):
                score = (s["q"][a:b, j].double() @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                lse[a:b, j] = score.logsumexp(-1)
                out[a:b, j] = score.softmax(-1) @ v
    return {"out": out, "lse": lse}
