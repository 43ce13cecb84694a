"""Plain 64-bit definitions of the serving operators (CPU, loops over sequences), and the batches
the tests run them on. Nothing here uses the library."""
import math

import torch

TYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16}


def half_step(t):
    """A rounding is off by at most this much of the value."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step among the smallest values of the type."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rope(x, weight, positions, table, interleaved, scale, eps):
    """x [tokens, heads, dim] in 64 bits, and a bound of the magnitudes that were added up."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    mag = y.abs().clone()
    if table is None:
        return y, mag
    y = y.clone()
    words = [int(w) % 2 ** 64 for w in table.tolist()]
    half = len(words)
    # p * w modulo one turn, exactly, then to 64-bit floating point
    turn = torch.tensor([[((int(p) * w) % 2 ** 64) / 2 ** 64 for w in words] for p in positions], dtype=torch.float64)
    cos, sin = (torch.cos(2 * math.pi * turn) * scale)[:, None], (torch.sin(2 * math.pi * turn) * scale)[:, None]
    i = torch.arange(half)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., a_at].clone(), y[..., b_at].clone()
    y[..., a_at], y[..., b_at] = a * cos - b * sin, b * cos + a * sin
    mag[..., a_at] = mag[..., b_at] = (a.abs() + b.abs()) * abs(scale)
    return y, mag


def check_rope(got, ref, mag, what):
    """One rounding to the type; before it the norm (sum of squares, root, two products: under 16
    roundings of 2^-24) and the rotation (angle within 1e-7 rad, cosine and sine within 2^-22, one
    product and one fma) stay within 2^-19 of the magnitudes added."""
    t = got.dtype
    got = got.double()
    assert torch.isfinite(got).all(), what
    bound = half_step(t) * ref.abs() * (1 + 2.0 ** -10) + 2.0 ** -19 * mag + tiny(t)
    worst = ((got - ref).abs() / bound).max()
    assert float(worst) <= 1.0, (what, float(worst))


def batch(n_q, kv, page_size, width=None, spare=2, prefix_pages=0, seed=0):
    """q_start, kv_lens, page_table, prefix pages and the number of pages, pages in a mixed order."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-k // page_size) for k in kv]
    width = max([1] + need) if width is None else width
    pages = sum(need) + prefix_pages + spare
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(kv), width), 2 ** 31 - 1, dtype=torch.int32)   # what is past the end is not read
    at = prefix_pages
    for s, w in enumerate(need):
        table[s, :w] = order[at : at + w]
        at += w
    q_start = torch.tensor([sum(n_q[:i]) for i in range(len(n_q) + 1)], dtype=torch.int32)
    return dict(q_start=q_start, kv_lens=torch.tensor(kv, dtype=torch.int32).reshape(len(kv)), page_table=table,
                prefix_pages=order[:prefix_pages].clone() if prefix_pages else None, pages=pages, page_size=page_size,
                n_q=list(n_q), kv=list(kv))


def keys_of(cache, b, s):
    """A sequence's keys (or values) with the shared prefix before them: [keys, heads, dim]; cache
    [pages, heads, rows, dim]."""
    ids = b["page_table"][s, : -(-b["kv"][s] // b["page_size"])]
    n = b["kv"][s]
    if b["prefix_pages"] is not None:
        ids = torch.cat((b["prefix_pages"], ids))
        n += len(b["prefix_pages"]) * b["page_size"]
    return cache[ids.long()].transpose(1, 2).flatten(0, 1)[:n]


def attention(q, k_cache, v_cache, b, scale, device="cpu"):
    """(out, lse, spread) in 64 bits; spread: sum p |v|, what the roundings of p are relative to."""
    tokens, hq, d = q.shape
    hk = k_cache.shape[1]
    g = hq // hk
    out = torch.zeros(tokens, hq, d, dtype=torch.float64)
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64)
    spread = torch.zeros_like(out)
    for s, n in enumerate(b["n_q"]):
        a = int(b["q_start"][s])
        k, v = (keys_of(x, b, s).to(device).double().transpose(0, 1) for x in (k_cache, v_cache))   # [hk, keys, d]
        count = k.shape[1]
        if n == 0 or count == 0:
            continue
        qq = q[a : a + n].to(device).double().view(n, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * n, d)
        score = (qq @ k.transpose(1, 2) * scale).view(hk, g, n, count)
        seen = torch.arange(count, device=device) < torch.arange(count - n + 1, count + 1, device=device)[:, None]
        score = score.masked_fill(~seen, -math.inf)
        some = seen.any(-1)   # [n]
        top = torch.where(some, score.amax(-1), torch.zeros((), dtype=torch.float64, device=device))
        p = torch.exp(score - top[..., None])
        total = p.sum(-1)
        p = p / torch.where(total > 0, total, torch.ones_like(total))[..., None]
        o = (p.view(hk, g * n, count) @ v).view(hk, g, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)
        w = (p.view(hk, g * n, count) @ v.abs()).view(hk, g, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)
        out[a : a + n], spread[a : a + n] = o.cpu(), w.cpu()
        lse[a : a + n] = torch.where(some, top + total.log(), -math.inf).permute(2, 0, 1).reshape(n, hq).cpu()
    return out, lse, spread


def check_attention(got, got_lse, ref, lse, spread, what):
    """The output's rounding; before it each probability's rounding to the type (half a step each,
    against the sum of the unrounded ones), scores off by at most 2^-18 (128 products of FP32 sums
    of magnitudes up to 40, an FP32 base-2 scaling and 2^x within 2^-22) and FP32 sums: together
    within half a step plus 2^-16 of sum p |v|."""
    t = got.dtype
    got, got_lse = got.double(), got_lse.double()
    assert torch.isfinite(got).all(), what
    bound = half_step(t) * ref.abs() * (1 + 2.0 ** -7) + (half_step(t) + 2.0 ** -16) * spread + tiny(t)
    worst = ((got - ref).abs() / bound).max()
    assert float(worst) <= 1.0, (what, float(worst))
    none = torch.isinf(lse)
    assert torch.equal(got_lse[none], lse[none]), what
    assert torch.all(got[none] == 0), what
    err = (got_lse - lse)[~none].abs()
    assert err.numel() == 0 or float((err / (2.0 ** -16 + 2.0 ** -22 * lse[~none].abs())).max()) <= 1.0, (what, float(err.max()))
