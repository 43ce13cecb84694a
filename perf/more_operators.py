"""Operators of decoding a few tokens at a time on a paged key/value cache: attention for trees of
drafted tokens, the accepted drafts taken over, a cache held to a bounded size by the attention
weight that its keys have drawn, and products with 4-bit weights for few rows. ``run`` computes
them in plain torch operations, or through the library when ``own`` is true; ``exact`` computes
them again in 64 bits.

Sequence s has the new tokens q_start[s] .. q_start[s + 1] - 1 of the flat token dimension and,
with them, kv_lens[s] keys in the pages page_table[s][0], page_table[s][1], ... of the cache; keys
of a shared prefix come before them. New token i of n has its key at place kv_len - n + i.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda:0"
_GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------------- the cases

def _cached(op, name, **kw):
    d = dict(name=name, op=op, dtype="float16", seqs=1, q_min=1, q_max=1, ctx_min=0, ctx_max=0, kv_heads=8, head_dim=128,
             page_size=16, by_rows=False)
    if op in ("tree", "weigh"):
        d.update(q_heads=32)
    if op == "tree":
        d.update(prefix_pages=0, roots=1)
    if op == "weigh":
        d.update(window=0, decay=1.0)
    if op == "evict":
        d.update(keep=1024, first=4, recent=64)
    if op == "accept":
        d.update(depth=4)
    d.update(kw)
    return d


def _w4(name, **kw):
    d = dict(name=name, op="w4", dtype="float16", rows=1, n=4096, k=4096, group=128, zeros=True, bias=False, act="none")
    d.update(kw)
    return d


def listed():
    return [
        # one user's five drafted tokens behind a short text: the latency of a call
        _cached("tree", "tree_one_user", q_min=5, q_max=5, ctx_min=776, ctx_max=776),
        # a verification step of 48 users with trees of up to 16 nodes, whose texts differ much in length
        _cached("tree", "tree_step", dtype="bfloat16", seqs=48, q_min=4, q_max=16, ctx_min=15, ctx_max=8191, page_size=64),
        # wide trees of 64 nodes behind very long texts: several tiles of rows, the keys split over the GPU
        _cached("tree", "tree_wide_far", seqs=3, q_min=63, q_max=64, ctx_min=90000, ctx_max=131000, page_size=256, roots=8),
        # after a decoding step of 64 users: the weight that the new tokens give to each key
        _cached("weigh", "weigh_step", dtype="bfloat16", seqs=64, ctx_min=15, ctx_max=8191, page_size=64),
        # after five prompts: the weight that the last 32 tokens of each give to all of its keys
        _cached("weigh", "weigh_window", seqs=5, q_min=300, q_max=8200, page_size=32, by_rows=True, window=32, decay=0.0),
        # one user's cache brought back to 1024 keys
        _cached("evict", "evict_one_user", ctx_min=1090, ctx_max=1090),
        # twelve long caches brought to 2048 keys each
        _cached("evict", "evict_many", dtype="bfloat16", seqs=12, ctx_min=3000, ctx_max=16000, page_size=64, keep=2048, recent=512),
        # the accepted path of 48 trees of 16 nodes
        _cached("accept", "accept_step", dtype="bfloat16", seqs=48, q_min=4, q_max=16, ctx_min=15, ctx_max=1000, page_size=64),
        # many users with wide trees, heads of 64, a token-major cache
        _cached("accept", "accept_many_d64", seqs=200, q_min=20, q_max=64, ctx_max=600, kv_heads=16, head_dim=64, by_rows=True,
                depth=12),
        # one token through a square projection: a matrix-vector product
        _w4("w4_token"),
        # eight tokens through the MLP benchmark's up-projection with its epilogue
        _w4("w4_mlp_up", rows=8, n=16384, bias=True, act="gelu"),
        # a step of 64 users through the down-projection, finer groups
        _w4("w4_mlp_down_users", dtype="bfloat16", rows=64, k=16384, group=64, zeros=False, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "weigh", "evict", "accept", "w4", "w4"])
    c = dict(op=op, dtype=rng.choice(["float16", "bfloat16"]))
    if op == "w4":
        group = rng.choice([32, 64, 128])
        n, k = 8 * _log(rng, 8, 2048), group * _log(rng, max(1, 256 // group), 16384 // group)
        while n * k > 16384 * 4096:
            n, k = 8 * (n // 16), group * max(1, k // (2 * group))
        c.update(rows=_log(rng, 1, 64), n=n, k=k, group=group, zeros=rng.random() < 0.6, bias=rng.random() < 0.5,
                 act=rng.choice(["none", "none", "gelu", "relu"]))
        return c
    head_dim, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 5, 8, 16])
    c.update(head_dim=head_dim, kv_heads=kv_heads, page_size=rng.choice([16, 32, 64, 128, 256]), by_rows=rng.random() < 0.5)
    room = 200000000 // (kv_heads * head_dim)   # keys of all sequences
    seqs = _log(rng, 1, 128)
    ctx_max = _log(rng, 16, min(100000, room // seqs))
    c.update(seqs=seqs, ctx_max=ctx_max, ctx_min=rng.randint(0, ctx_max), q_min=1, q_max=1)
    if op in ("tree", "weigh"):
        c.update(q_heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8]))
    if op in ("tree", "accept"):
        q_max = _log(rng, 1, 64)
        if op == "tree":   # the plain form holds all scores
            q_max = max(1, min(q_max, 700000000 // (seqs * c["q_heads"] * ctx_max)))
        c.update(q_max=q_max, q_min=rng.randint(1, q_max))
    if op == "tree":
        c.update(prefix_pages=0 if rng.random() < 0.6 else _log(rng, 1, 64), roots=rng.randint(1, 8))
    if op == "accept":
        c.update(depth=rng.randint(1, 16))
    if op == "evict":
        first, recent = rng.choice([0, 1, 4]), _log(rng, 1, 512)
        c.update(first=first, recent=recent, keep=first + recent + _log(rng, 1, 4096), ctx_min=max(1, c["ctx_min"]))
    if op == "weigh":
        if rng.random() < 0.4:   # prompts, or pieces of them
            q_max = min(_log(rng, 8, 4096), ctx_max)
            window = min(q_max, _log(rng, 1, 64))
            c.update(q_max=q_max, q_min=rng.randint(1, q_max), window=window, decay=rng.choice([0.0, 0.5, 1.0]))
            while c["seqs"] * (ctx_max + q_max) * c["q_heads"] * window > 700000000:
                c["seqs"] = (c["seqs"] + 1) // 2
                if c["seqs"] == 1:
                    break
        else:
            c.update(window=0, decay=rng.choice([1.0, 0.9]))
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
    """New tokens and keys (the new ones among them) of each sequence; an eviction has no new tokens."""
    ctx = _spread(c["seqs"], c["ctx_min"], c["ctx_max"], 0.0)
    if c["op"] == "evict":
        return [0] * c["seqs"], ctx
    n_q = _spread(c["seqs"], c["q_min"], c["q_max"], 0.3)
    return n_q, [a + b for a, b in zip(n_q, ctx)]


# ---------------------------------------------------------------------------------- the inputs

def _trees(n_q, roots, gen):
    """A parent for each node: one of the few before it, or -1 for the first `roots` nodes."""
    parents = []
    for n in n_q:
        u = torch.rand(n, generator=gen).tolist()
        parents += [-1 if i < roots else max(0, i - 1 - int(u[i] * 12)) for i in range(n)]
    return parents


def _paths(n_q, depth, gen):
    """Accepted nodes of each tree, from the root on: ascending, one at least."""
    index, counts = torch.zeros(len(n_q), depth, dtype=torch.int32), []
    for s, n in enumerate(n_q):
        u = torch.rand(depth, generator=gen).tolist()
        node, path = -1, []
        for j in range(1 + int(u[0] * min(depth, n))):
            node += 1 + int(u[j] * 3)
            if node >= n:
                break
            path.append(node)
        path = path or [0]
        index[s, : len(path)] = torch.tensor(path, dtype=torch.int32)
        counts.append(len(path))
    return index, torch.tensor(counts, dtype=torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = getattr(torch, c["dtype"])

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32) * scale).to(dt)

    s = dict(case=dict(c))
    if c["op"] == "w4":
        n, k, groups = c["n"], c["k"], c["k"] // c["group"]
        s["a"] = normal(c["rows"], k)
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=gen, device=DEVICE, dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand(n, groups, generator=gen, device=DEVICE)) * 0.2 / math.sqrt(k)).to(dt)
        s["zeros"] = torch.randint(6, 11, (n, groups), generator=gen, device=DEVICE, dtype=torch.uint8) if c["zeros"] else None
        s["bias"] = normal(n, scale=0.1) if c["bias"] else None
        return s
    host = torch.Generator().manual_seed(int(seed))
    n_q, kv = _lengths(c)
    hk, d, ps, n = c["kv_heads"], c["head_dim"], c["page_size"], c["seqs"]
    prefix = c.get("prefix_pages", 0)
    need = [-(-x // ps) for x in kv]
    pages = sum(need) + prefix + 2
    order = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.zeros(n, max(need), dtype=torch.int32)
    at = prefix
    for i, w in enumerate(need):
        table[i, :w] = order[at : at + w]
        at += w
    s["page_table"] = table.to(DEVICE)
    s["prefix_pages"] = order[:prefix].to(DEVICE) if prefix else None
    s["q_start"] = torch.tensor(np.cumsum([0] + n_q), dtype=torch.int32, device=DEVICE)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEVICE)
    s["max_q"], s["max_kv"], s["tokens"] = max(n_q), max(kv), sum(n_q)
    shape = (pages, ps, hk, d) if c["by_rows"] else (pages, hk, ps, d)
    cache = [normal(*shape) for _ in range(2)]
    s["k_cache"], s["v_cache"] = [x.transpose(1, 2) if c["by_rows"] else x for x in cache]   # [page, head, row, dim]
    if c["op"] in ("weigh", "evict"):
        # heavy tails, and some keys that nothing has looked at
        w = torch.exp(2 * torch.randn(pages, hk, ps, generator=gen, device=DEVICE))
        s["weights"] = w * (torch.rand(pages, hk, ps, generator=gen, device=DEVICE) > 0.1)
    if c["op"] in ("tree", "weigh"):
        s["q"] = normal(s["tokens"], c["q_heads"], d)
    if c["op"] == "tree":
        s["parents"] = torch.tensor(_trees(n_q, c["roots"], host), dtype=torch.int32, device=DEVICE)
    if c["op"] == "weigh":   # as the attention of these tokens has left it
        s["lse"] = torch.zeros(s["tokens"], c["q_heads"], device=DEVICE)
        score, token, on = _window_scores(s)
        s["lse"][token[on]] = torch.logsumexp(score, -1).permute(0, 3, 1, 2).flatten(2)[on]
    if c["op"] == "accept":
        index, counts = _paths(n_q, c["depth"], host)
        s["index"], s["counts"] = index.to(DEVICE), counts.to(DEVICE)
        s["start"] = s["kv_lens"] - torch.tensor(n_q, dtype=torch.int32, device=DEVICE)
    return s


# ------------------------------------------------------------------------------ the plain form

def _keys(cache, pages):
    """[..., pages] -> [..., heads, keys, dim] in 32 bits."""
    return cache[pages.long()].float().transpose(-4, -3).flatten(-3, -2)


def _plain_tree(s):
    c = s["case"]
    hq, hk, d, ps, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["page_size"], c["seqs"]
    g, mq, tokens = hq // hk, s["max_q"], s["tokens"]
    prefix = c["prefix_pages"] * ps
    q_start, kv_lens = s["q_start"].long(), s["kv_lens"].long()
    n_q = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=DEVICE)
    on = i < n_q[:, None]
    token = (q_start[:-1, None] + i).clamp(max=tokens - 1)                     # [n, mq]
    # ancestors: the powers of (1 + the step to the parent)
    step = (s["parents"].long()[token][..., None] == i) & on[..., None]        # [n, node, parent]
    seen = torch.matrix_power(step.float() + torch.eye(mq, device=DEVICE), mq) > 0.5
    seen = seen & on[..., None]                                                # (rows of padding: none)
    words = -(-mq // 32)
    bits = torch.zeros(n, mq, 32 * words, dtype=torch.int64, device=DEVICE)
    bits[..., :mq] = seen
    word = (bits.view(n, mq, words, 32) << torch.arange(32, device=DEVICE)).sum(-1)
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()
    place = (prefix + kv_lens - n_q)[:, None] + seen.sum(-1) - 1

    q = s["q"].float()[token].view(n, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * mq, d)
    k, v = _keys(s["k_cache"], s["page_table"]), _keys(s["v_cache"], s["page_table"])
    at = torch.arange(k.shape[2], device=DEVICE)
    v = v * (at < kv_lens[:, None])[:, None, :, None]
    node = at - (kv_lens - n_q)[:, None]                                       # [n, keys]
    own_keys = torch.gather(seen, 2, node.clamp(0, mq - 1)[:, None].expand(n, mq, -1)) & (node < n_q[:, None])[:, None]
    visible = (node < 0)[:, None] | own_keys                                   # [n, mq, keys]
    score = (q @ k.transpose(-1, -2)).view(n, hk, g, mq, -1) * (1.0 / math.sqrt(d))
    score = score.masked_fill(~visible[:, None, None], -math.inf)
    if prefix:
        kp, vp = _keys(s["k_cache"], s["prefix_pages"]), _keys(s["v_cache"], s["prefix_pages"])
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
    to = torch.where(on, token, tokens)

    def flat(x, dtype):
        y = torch.empty(tokens + 1, *x.shape[2:], device=DEVICE, dtype=dtype)
        y[to] = x.to(dtype)
        return y[:tokens]

    return {"out": flat(o, s["q"].dtype), "lse": flat(lse, torch.float32), "mask": flat(word, torch.int32),
            "positions": flat(place, torch.int32)}


def _window_scores(s):
    """Scaled scores of the tokens in the window [seqs, key heads, heads of a group, tokens, keys] (-inf: not seen),
    those tokens [seqs, tokens] and whether there are so many."""
    c = s["case"]
    hq, hk, d, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["seqs"]
    g = hq // hk
    q_start, kv_lens = s["q_start"].long(), s["kv_lens"].long()
    n_q = q_start[1:] - q_start[:-1]
    w = min(c["window"] or s["max_q"], s["max_q"])
    back = torch.arange(w, device=DEVICE) - w                      # -w .. -1: counted from the last token
    on = back >= -n_q[:, None]
    token = (q_start[1:, None] + back).clamp(min=0)
    q = s["q"].float()[token].view(n, w, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * w, d)
    k = _keys(s["k_cache"], s["page_table"])
    score = (q @ k.transpose(-1, -2)).view(n, hk, g, w, -1) * (1.0 / math.sqrt(d))
    hidden = torch.arange(k.shape[2], device=DEVICE) > (kv_lens[:, None] + back)[..., None]
    return score.masked_fill((hidden | ~on[..., None])[:, None, None], -math.inf), token, on


def _plain_weigh(s):
    c = s["case"]
    ps, n = c["page_size"], c["seqs"]
    g = c["q_heads"] // c["kv_heads"]
    score, token, on = _window_scores(s)
    lse = s["lse"][token].view(n, -1, c["kv_heads"], g).permute(0, 2, 3, 1)[..., None]
    add = torch.exp(score - lse).sum((2, 3))                       # [n, heads, keys]
    q_start, kv_lens = s["q_start"].long(), s["kv_lens"].long()
    at = torch.arange(add.shape[-1], device=DEVICE)
    page = s["page_table"].long()[:, at // ps]                     # [n, keys]
    row = (at % ps).expand(n, -1)
    heads = torch.arange(c["kv_heads"], device=DEVICE)[None, :, None]
    old = s["weights"][page[:, None], heads, row[:, None]]
    new_key = at >= (kv_lens - (q_start[1:] - q_start[:-1]))[:, None]
    w = torch.where(new_key[:, None], add, old * c["decay"] + add)
    # keys past a sequence's end: its first key again, as it is
    there = at < kv_lens[:, None]
    page, row = torch.where(there, page, page[:, :1]), torch.where(there, row, row[:, :1])
    s["weights"][page[:, None], heads, row[:, None]] = torch.where(there[:, None], w, w[..., :1])
    return {"weights": s["weights"]}


def _move(s, index, counts, start, weights):
    """Row start + j <- row start + index[j] for j < counts; index [n, heads, most]. Entries past a count repeat the first."""
    c = s["case"]
    ps, most = c["page_size"], index.shape[-1]
    j = torch.arange(most, device=DEVICE).expand_as(index)
    on = j < counts.long()[:, None, None]
    start = start.long()[:, None, None]
    src, dst = start + torch.where(on, index.long(), index[..., :1].long()), start + torch.where(on, j, 0)
    seq = torch.arange(c["seqs"], device=DEVICE)[:, None, None]
    heads = torch.arange(c["kv_heads"], device=DEVICE)[None, :, None]
    table = s["page_table"].long()
    src, dst = (table[seq, src // ps], heads, src % ps), (table[seq, dst // ps], heads, dst % ps)
    for x in (s["k_cache"], s["v_cache"]) + ((weights,) if weights is not None else ()):
        x[dst] = x[src]


def _plain_evict(s):
    c = s["case"]
    ps, n, hk, keep = c["page_size"], c["seqs"], c["kv_heads"], c["keep"]
    kv = s["kv_lens"].long()[:, None, None]
    at = torch.arange(max(s["max_kv"], keep), device=DEVICE)
    page = s["page_table"].long()[:, (at // ps).clamp(max=s["page_table"].shape[1] - 1)]
    heads = torch.arange(hk, device=DEVICE)[None, :, None]
    w = s["weights"][page[:, None], heads, (at % ps)[None, None]]
    w = torch.where((at < c["first"]) | (at >= kv - c["recent"]), math.inf, w)
    w = torch.where(at < kv, w, -math.inf)
    picked = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    counts = s["kv_lens"].clamp(max=keep)
    on = torch.arange(keep, device=DEVICE) < counts[:, None, None]
    picked = torch.sort(torch.where(on, picked, at.shape[0])).values
    index = torch.where(on, picked, -1).int()
    _move(s, index, counts, torch.zeros_like(counts), s["weights"])
    return {"index": index, "lens": counts, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"]}


def _plain_accept(s):
    index = s["index"][:, None].expand(-1, s["case"]["kv_heads"], -1)
    _move(s, index, s["counts"], s["start"], None)
    return {"lens": s["start"] + s["counts"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_w4(s):
    c = s["case"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).flatten(1)     # the even column in the low half
    zeros = s["zeros"].float()[..., None] if s["zeros"] is not None else 8.0
    w = (codes.float().view(c["n"], -1, c["group"]) - zeros) * s["scales"].float()[..., None]
    y = s["a"].float() @ w.flatten(1).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "gelu":
        y = y * 0.5 * (1 + torch.erf(y * math.sqrt(0.5)))
    if c["act"] == "relu":
        y = y.clamp(min=0)
    return {"c": y.to(s["a"].dtype)}


# ------------------------------------------------------------------------- the library's calls

_context = None


def _library():
    global _context
    import tensor_core_gemm_tcgen05_gb300 as g
    if _context is None:
        _context = g.Context(0)
    return g, _context


def _own_tree(s):
    g, ctx = _library()
    c = s["case"]
    mask, positions = g.tree_mask(ctx, s["parents"], s["q_start"], s["kv_lens"], s["max_q"],
                                  prefix_len=c["prefix_pages"] * c["page_size"])
    lse = torch.empty(s["tokens"], c["q_heads"], dtype=torch.float32, device=DEVICE)
    out = g.tree_attention(ctx, s["q"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_lens"], s["page_table"], mask,
                           max_q=s["max_q"], prefix_pages=s["prefix_pages"], lse=lse)
    return {"out": out, "lse": lse, "mask": mask, "positions": positions}


def _own_weigh(s):
    g, ctx = _library()
    c = s["case"]
    w = g.kv_weigh(ctx, s["q"], s["k_cache"], s["q_start"], s["kv_lens"], s["page_table"], s["lse"], s["weights"],
                   window=c["window"], decay=c["decay"])
    return {"weights": w}


def _own_evict(s):
    g, ctx = _library()
    c = s["case"]
    index, counts = g.kv_select(ctx, s["weights"], s["kv_lens"], s["page_table"], c["keep"], first=c["first"], recent=c["recent"])
    lens = g.kv_compact(ctx, s["k_cache"], s["v_cache"], s["kv_lens"], s["page_table"], index, counts, weights=s["weights"])
    return {"index": index, "lens": lens, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"]}


def _own_accept(s):
    g, ctx = _library()
    lens = g.kv_compact(ctx, s["k_cache"], s["v_cache"], s["kv_lens"], s["page_table"], s["index"], s["counts"], start=s["start"])
    return {"lens": lens, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_w4(s):
    g, ctx = _library()
    act = {"none": g.EPI_NONE, "gelu": g.EPI_GELU, "relu": g.EPI_RELU}[s["case"]["act"]]
    return {"c": g.w4_gemm(ctx, s["a"], s["codes"], s["scales"], s["zeros"], bias=s["bias"], epilogue=act)}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "weigh": _own_weigh, "evict": _own_evict, "accept": _own_accept, "w4": _own_w4}[op](state)
    return {"tree": _plain_tree, "weigh": _plain_weigh, "evict": _plain_evict, "accept": _plain_accept, "w4": _plain_w4}[op](state)


# ------------------------------------------------------------------------- what a pass has to do

def work(case):
    c = case
    if c["op"] == "w4":
        m, n, k = c["rows"], c["n"], c["k"]
        groups = n * (k // c["group"])
        return {"bytes": n * k // 2 + groups * (3 if c["zeros"] else 2) + 2 * m * (n + k) + (2 * n if c["bias"] else 0),
                "flops": 2 * m * n * k}
    n_q, kv = _lengths(c)
    hk, d, ps = c["kv_heads"], c["head_dim"], c["page_size"]
    tables = 4 * sum(-(-k // ps) for k in kv) + 8 * c["seqs"]
    t, keys = sum(n_q), sum(kv)
    if c["op"] == "tree":
        prefix = c["prefix_pages"] * ps
        seen = sum(n * (prefix + k - n) + n for n, k in zip(n_q, kv))   # (every node sees itself, most a few more)
        return {"bytes": 4 * t * c["q_heads"] * d + 4 * t * c["q_heads"] + 4 * (keys + prefix) * hk * d + tables
                + t * (8 + 4 * -(-max(n_q) // 32)), "flops": 4 * d * c["q_heads"] * seen}
    if c["op"] == "weigh":
        rows = [min(n, c["window"] or n) for n in n_q]
        seen = sum(r * k - r * (r - 1) // 2 for r, k in zip(rows, kv))
        old = 0 if c["decay"] == 0.0 else sum(k - n for n, k in zip(n_q, kv))
        return {"bytes": sum(rows) * c["q_heads"] * (2 * d + 4) + 2 * keys * hk * d + 4 * hk * (old + keys) + tables,
                "flops": 2 * d * c["q_heads"] * seen}
    if c["op"] == "evict":   # (the first rows stay where they are)
        moved = sum(c["keep"] - c["first"] for k in kv if k > c["keep"])
        kept = sum(min(k, c["keep"]) for k in kv)
        return {"bytes": 4 * keys * hk + 4 * kept * hk + moved * hk * (8 * d + 8) + tables, "flops": 0}
    moved = sum(min(c["depth"], n) for n in n_q) // 2
    return {"bytes": moved * hk * 8 * d + 4 * moved + 16 * c["seqs"], "flops": 0}


# --------------------------------------------------------------------------- in 64 bits, apart

def _own_rows(s, cache, i, count):
    """Keys 0 .. count - 1 of sequence i: [heads, keys, dim] in 64 bits."""
    ps = s["case"]["page_size"]
    at = torch.arange(count, device=DEVICE)
    return cache[s["page_table"][i].long()[at // ps], :, at % ps].double().transpose(0, 1)


def _exact_tree(s, n_q, kv):
    c = s["case"]
    hq, hk, d, g = c["q_heads"], c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    prefix = c["prefix_pages"] * c["page_size"]
    out = torch.empty(s["tokens"], hq, d, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["tokens"], hq, dtype=torch.float64, device=DEVICE)
    masks, positions = np.zeros((s["tokens"], -(-s["max_q"] // 32)), np.uint32), []
    parents = s["parents"].tolist()
    a = 0
    for i in range(c["seqs"]):
        n, total = n_q[i], prefix + kv[i]
        line = []   # the path of each node
        for j in range(n):
            up = parents[a + j]
            line.append((line[up] if up >= 0 else []) + [j])
            for x in line[j]:
                masks[a + j, x // 32] |= np.uint32(1 << (x % 32))
            positions.append(total - n + len(line[j]) - 1)
        hidden = torch.ones(n, total, dtype=torch.bool)
        hidden[:, : total - n] = False
        for j in range(n):
            hidden[j, [total - n + x for x in line[j]]] = False
        hidden = hidden.to(DEVICE)
        k, v = _own_rows(s, s["k_cache"], i, kv[i]), _own_rows(s, s["v_cache"], i, kv[i])
        if prefix:
            k, v = [torch.cat((x[s["prefix_pages"].long()].double().transpose(0, 1).flatten(1, 2), y), 1)
                    for x, y in ((s["k_cache"], k), (s["v_cache"], v))]
        for h in range(hq):
            score = (s["q"][a : a + n, h].double() @ k[h // g].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[a : a + n, h] = score.logsumexp(-1)
            out[a : a + n, h] = score.softmax(-1) @ v[h // g]
        a += n
    return {"out": out, "lse": lse, "mask": torch.from_numpy(masks.view(np.int32)),
            "positions": torch.tensor(positions, dtype=torch.int32)}


def _exact_weigh(s, n_q, kv):
    c = s["case"]
    ps, g, d = c["page_size"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    weights = s["weights"].double()
    end = 0
    for i in range(c["seqs"]):
        end += n_q[i]
        rows = min(n_q[i], c["window"] or n_q[i])
        k = _own_rows(s, s["k_cache"], i, kv[i])
        at = torch.arange(kv[i], device=DEVICE)
        hidden = at > torch.arange(kv[i] - rows, kv[i], device=DEVICE)[:, None]
        page = s["page_table"][i].long()[at // ps]
        factor = torch.where(at < kv[i] - n_q[i], c["decay"], 0.0).double()
        for h in range(c["kv_heads"]):
            w = weights[page, h, at % ps] * factor
            for j in range(h * g, (h + 1) * g):
                score = s["q"][end - rows : end, j].double() @ k[h].T / math.sqrt(d) - s["lse"][end - rows : end, j, None].double()
                w = w + score.masked_fill(hidden, -math.inf).exp().sum(0)
            weights[page, h, at % ps] = w
    return {"weights": weights}


def _exact_rows(s, i, h, index, at, what):
    """Rows of one sequence and head gathered, then written in order."""
    ps, table = s["case"]["page_size"], s["page_table"][i].long()
    index = torch.as_tensor(index, device=DEVICE).long() + at
    to = torch.arange(at, at + index.shape[0], device=DEVICE)
    for x in what:
        x[table[to // ps], h, to % ps] = x[table[index // ps], h, index % ps].clone()


def _exact_evict(s, kv):
    c = s["case"]
    ps, hk = c["page_size"], c["kv_heads"]
    index, lens = np.full((c["seqs"], hk, c["keep"]), -1, np.int32), []
    moved = [s["k_cache"].double(), s["v_cache"].double(), s["weights"].double()]
    weights, table = s["weights"].cpu().numpy(), s["page_table"].cpu().numpy()
    for i in range(c["seqs"]):
        lens.append(min(kv[i], c["keep"]))
        at = np.arange(kv[i])
        for h in range(hk):
            w = weights[table[i, at // ps], h, at % ps]
            kept = at
            if kv[i] > c["keep"]:
                middle = at[c["first"] : kv[i] - c["recent"]]
                best = middle[np.lexsort((middle, -w[middle]))][: c["keep"] - c["first"] - c["recent"]]
                kept = np.sort(np.concatenate((at[: c["first"]], best, at[kv[i] - c["recent"] :])))
            index[i, h, : lens[-1]] = kept
            _exact_rows(s, i, h, kept, 0, moved)
    return {"index": torch.from_numpy(index), "lens": torch.tensor(lens, dtype=torch.int32), "k_cache": moved[0], "v_cache": moved[1],
            "weights": moved[2]}


def _exact_accept(s):
    moved = [s["k_cache"].double(), s["v_cache"].double()]
    counts, start = s["counts"].tolist(), s["start"].tolist()
    for i in range(s["case"]["seqs"]):
        _exact_rows(s, i, slice(None), s["index"][i, : counts[i]], start[i], moved)
    return {"lens": torch.tensor([a + b for a, b in zip(start, counts)], dtype=torch.int32), "k_cache": moved[0], "v_cache": moved[1]}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "w4":
        w = torch.empty(c["n"], c["k"], dtype=torch.float64, device=DEVICE)
        w[:, 0::2], w[:, 1::2] = s["codes"] % 16, s["codes"] // 16
        w -= s["zeros"].double().repeat_interleave(c["group"], 1) if c["zeros"] else 8
        y = s["a"].double() @ (w * s["scales"].double().repeat_interleave(c["group"], 1)).T
        y = y + (s["bias"].double() if c["bias"] else 0)
        return {"c": y * torch.special.ndtr(y) if c["act"] == "gelu" else torch.relu(y) if c["act"] == "relu" else y}
    n_q, kv = _lengths(c)
    if work(c)["flops"] > 4e12:
        return None
    if c["op"] == "tree":
        return _exact_tree(s, n_q, kv)
    if c["op"] == "weigh":
        return _exact_weigh(s, n_q, kv)
    return _exact_evict(s, kv) if c["op"] == "evict" else _exact_accept(s)
