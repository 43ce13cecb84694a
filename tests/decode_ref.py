"""Plain 64-bit definitions of the operators of include/gemm_decode.h (CPU, loops), and the inputs
the tests run them on. Nothing here uses the library."""
import math

import torch

from serving_ref import half_step, keys_of, tiny


def trees(n_q, seed=0, reach=6, roots=2):
    """parents of random trees, one per token."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for n in n_q:
        for i in range(n):
            u = float(torch.rand(1, generator=gen))
            out.append(-1 if i < roots else max(0, i - 1 - int(u * reach)))
    return torch.tensor(out, dtype=torch.int32)


def path(parents, a, i):
    """Nodes from i up to its root, in a tree whose first token is a."""
    line = []
    while i >= 0:
        line.append(i)
        i = int(parents[a + i])
    return line


def tree_mask(parents, b, words, prefix=0):
    """(mask int32 [tokens, words], positions int32) of a batch."""
    tokens = len(parents)
    mask = torch.zeros(tokens, words, dtype=torch.int64)
    positions = torch.zeros(tokens, dtype=torch.int32)
    for s, n in enumerate(b["n_q"]):
        a = int(b["q_start"][s])
        for i in range(n):
            line = path(parents, a, i)
            for j in line:
                mask[a + i, j // 32] |= 1 << (j % 32)
            positions[a + i] = prefix + b["kv"][s] - n + len(line) - 1
    return signed(mask), positions


def signed(words):
    """32-bit words, given as non-negative 64-bit integers, as int32."""
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()


def visible(mask, b, s, count):
    """[new tokens, keys of a sequence with its prefix]: whether the token sees the key."""
    n, a = b["n_q"][s], int(b["q_start"][s])
    bits = (mask[a : a + n].long()[..., None] >> torch.arange(32)) & 1
    bits = bits.flatten(1)[:, :n].bool()
    bits = torch.cat((bits, torch.zeros(n, max(0, n - bits.shape[1]), dtype=torch.bool)), 1)
    return torch.cat((torch.ones(n, count - n, dtype=torch.bool), bits), 1)


def tree_attention(q, k_cache, v_cache, b, mask, scale):
    """(out, lse, spread) in 64 bits; spread: sum p |v|."""
    tokens, hq, d = q.shape
    hk = k_cache.shape[1]
    g = hq // hk
    out = torch.zeros(tokens, hq, d, dtype=torch.float64)
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64)
    spread = torch.zeros_like(out)
    for s, n in enumerate(b["n_q"]):
        a = int(b["q_start"][s])
        k, v = (keys_of(x, b, s).double().transpose(0, 1) for x in (k_cache, v_cache))   # [hk, keys, d]
        count = k.shape[1]
        if n == 0 or count == 0:
            continue
        see = visible(mask, b, s, count)
        for h in range(hq):
            for i in range(n):
                on = see[i]
                if not on.any():
                    continue
                score = k[h // g][on] @ q[a + i, h].double() * scale
                lse[a + i, h] = torch.logsumexp(score, 0)
                p = torch.softmax(score, 0)
                out[a + i, h] = p @ v[h // g][on]
                spread[a + i, h] = p @ v[h // g][on].abs()
    return out, lse, spread


def weigh(q, k_cache, b, lse, weights, scale, window, decay):
    """(new weights, bound of their error) in 64 bits."""
    hk, ps = k_cache.shape[1], b["page_size"]
    g = q.shape[1] // hk
    w, bound = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    for s, n in enumerate(b["n_q"]):
        end, kv = int(b["q_start"][s]) + n, b["kv"][s]
        if kv == 0 or n == 0:   # (without new tokens: as it is)
            continue
        rows = min(n, window) if window else n
        k = keys_of(k_cache, {**b, "prefix_pages": None}, s).double()   # [keys, hk, d]
        at = torch.arange(kv)
        page, row = b["page_table"][s].long()[at // ps], at % ps
        for h in range(hk):
            add, slack = torch.zeros(kv, dtype=torch.float64), torch.zeros(kv, dtype=torch.float64)
            for i in range(n - rows, n):
                t, last = end - n + i, kv - n + i
                for j in range(h * g, (h + 1) * g):
                    if lse[t, j] == -math.inf or last < 0:
                        continue
                    x = k[: last + 1, h] @ q[t, j].double() * scale - lse[t, j].double()
                    p = torch.exp(x)
                    add[: last + 1] += p
                    # The exponent: scores within 2^-18 (as in serving_ref.check_attention), lse in base 2 rounded to
                    # 24 bits twice (the product, the sum with the score): 2^-23 of it; 2^x within 2^-22.
                    slack[: last + 1] += p * (2.0 ** -17 + 2.0 ** -23 * abs(float(lse[t, j])))
            old = torch.where(at < kv - n, w[page, h, row] * decay if decay else torch.zeros(kv, dtype=torch.float64),
                              torch.zeros(kv, dtype=torch.float64))
            w[page, h, row] = old + add
            # the FP32 sum: a rounding for each addition, of at most the total
            bound[page, h, row] = slack + (rows * g + 4) * 2.0 ** -24 * (old + add)
    return w, bound


def select(weights, kv, table, page_size, keep, first, recent):
    """index [seqs, heads, keep] (-1 behind the last), counts."""
    hk = weights.shape[1]
    index = torch.full((len(kv), hk, keep), -1, dtype=torch.int32)
    for s, n in enumerate(kv):
        for h in range(hk):
            kept = list(range(n))
            if n > keep:
                at = torch.arange(n)
                w = weights[table[s].long()[at // page_size], h, at % page_size].tolist()
                middle = range(first, n - recent)
                rank = sorted(middle, key=lambda i: (w[i] != w[i], -w[i] if w[i] == w[i] else 0, i))
                kept = sorted(list(range(first)) + rank[: keep - first - recent] + list(range(n - recent, n)))
            index[s, h, : len(kept)] = torch.tensor(kept, dtype=torch.int32)
    return index, torch.tensor([min(n, keep) for n in kv], dtype=torch.int32).reshape(len(kv))


def compact(arrays, table, page_size, index, counts, start):
    """Clones of arrays [pages, heads, rows, ...] with rows start + index[s][h][j] at start + j."""
    out = [x.clone() for x in arrays]
    for s in range(len(counts)):
        n, a = int(counts[s]), 0 if start is None else int(start[s])
        if n == 0:
            continue
        for h in range(arrays[0].shape[1]):
            src = a + (index[s, h] if index.dim() == 3 else index[s])[:n].long()
            dst = a + torch.arange(n)
            t = table[s].long()
            for x, y in zip(arrays, out):
                y[t[dst // page_size], h, dst % page_size] = x[t[src // page_size], h, src % page_size]
    return out


def gelu(x):
    return x * torch.special.ndtr(x)


def w4(a, codes, scales, zeros, bias, act):
    """(result in 64 bits, bound of the library's error before it is rounded)."""
    n, k = scales.shape[0], a.shape[1]
    if k:
        group = k // scales.shape[1]
        c = torch.stack((codes % 16, codes // 16), -1).flatten(1).double()
        z = 8.0 if zeros is None else (zeros % 16).double().repeat_interleave(group, 1)
        w = (c - z) * scales.double().repeat_interleave(group, 1)
        y, mag = a.double() @ w.T, a.double().abs() @ w.abs().T
        # A group's products are exact, their FP32 sum takes up to `group` additions off by 2^-23 of the magnitudes
        # each (the tensor cores may cut instead of rounding), and the groups' sums as many again, scaled.
        slack = mag * 2.0 ** -23 * (group + k // group + 16)
    else:
        y, slack = torch.zeros(a.shape[0], n, dtype=torch.float64), 0.0
    if bias is not None:
        y = y + bias.double()
        slack = slack + 2.0 ** -23 * y.abs()
    if act == "gelu":   # |gelu'| < 1.13; the error function by 7.1.26 of Abramowitz & Stegun, within 1.5e-7, and FP32 arithmetic
        y, slack = gelu(y), 1.13 * slack + 3e-7 * (1 + y.abs())
    if act == "relu":
        y = y.clamp(min=0)
    return y, slack


def check_w4(got, ref, slack, what):
    t = got.dtype
    bound = half_step(t) * ref.abs() * (1 + 2.0 ** -10) + slack * (1 + half_step(t)) + tiny(t)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), what
    assert bool((err <= bound).all()), (what, float((err / bound).max()))
