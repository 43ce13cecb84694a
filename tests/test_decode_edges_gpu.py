"""The operators of include/gemm_decode.h at the ends of what their calls allow: what is computed where a batch does not fit its mask or
its keys, the largest groups of heads, products with a single group of columns."""
import math

import pytest
import torch

import decode_ref as ref
import tensor_core_gemm_tcgen05_gb300 as g
from serving_ref import TYPES, attention, batch, check_attention, keys_of
from test_decode_gpu import cache_of, clean, complains, normal, on_gpu, w4_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    with g.Context(0) as c:
        yield c


def limited_tree_attention(q, k_cache, v_cache, b, mask, scale):
    """tree_attention of decode_ref for sequences with more new tokens than bits or than own keys: a token sees the prefix, the keys
    before the new ones, and own key (kv - n, 0 at least) + j where there is one and its bit j is set."""
    tokens, hq, d = q.shape
    hk = k_cache.shape[1]
    out, spread = torch.zeros(tokens, hq, d, dtype=torch.float64), torch.zeros(tokens, hq, d, dtype=torch.float64)
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64)
    for s, n in enumerate(b["n_q"]):
        k, v = (keys_of(x, b, s).double().transpose(0, 1) for x in (k_cache, v_cache))
        count, news = k.shape[1], min(n, b["kv"][s])
        for i in range(n):
            t = int(b["q_start"][s]) + i
            bits = ((mask[t].long()[:, None] >> torch.arange(32)) & 1).flatten().bool()
            bits = torch.cat((bits, torch.zeros(max(0, news - len(bits)), dtype=torch.bool)))[:news]
            see = torch.cat((torch.ones(count - news, dtype=torch.bool), bits))
            if not see.any():
                continue
            for h in range(hq):
                score = k[h * hk // hq][see] @ q[t, h].double() * scale
                lse[t, h] = torch.logsumexp(score, 0)
                p = torch.softmax(score, 0)
                out[t, h], spread[t, h] = p @ v[h * hk // hq][see], p @ v[h * hk // hq][see].abs()
    return out, lse, spread


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n_q,kv,words,prefix", [
    ([40], [100], 1, 0), ([40, 3], [40, 9], 1, 2), ([140], [700], 2, 0),       # nodes past the mask
    ([8], [5], 1, 0), ([8, 30], [5, 300], 1, 1), ([50], [20], 2, 0),           # more nodes than keys
    ([8], [0], 1, 0), ([8], [0], 1, 1), ([1, 9, 2], [4, 0, 2], 1, 0),          # no keys of their own
    ([100], [70], 1, 1)])                                                      # both
def test_what_does_not_fit_is_reported_and_limited(ctx, dtype, n_q, kv, words, prefix):
    dt, hq, hk, d, ps = TYPES[dtype], 8, 2, 64, 16
    b = batch(n_q, kv, ps, prefix_pages=prefix, seed=1)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    q = normal(sum(n_q), hq, d, seed=3, dtype=dt)
    gen = torch.Generator().manual_seed(4)
    mask = ref.signed(torch.randint(0, 2 ** 32, (sum(n_q), words), generator=gen) | (torch.arange(sum(n_q)) % 3 == 0)[:, None].long())
    mask[-1] = 0
    lse = torch.empty(sum(n_q), hq, device="cuda")
    out = g.tree_attention(ctx, q.cuda(), kd, vd, *on_gpu(b).values(), mask.cuda(), lse=lse,
                           prefix_pages=b["prefix_pages"].cuda() if prefix else None)
    complains(ctx)
    check_attention(out.cpu(), lse.cpu(), *limited_tree_attention(q, k, v, b, mask, 1 / math.sqrt(d)), (dtype, n_q, kv, words, prefix))


@pytest.mark.parametrize("n,kv,words", [(70, 90, 2), (2048 + 5, 2100, 64)])
def test_nodes_past_the_mask_get_no_bits(ctx, n, kv, words):
    b = batch([n], [kv], 16)
    parents = torch.arange(-1, n - 1, dtype=torch.int32)
    mask, positions = g.tree_mask(ctx, parents.cuda(), b["q_start"].cuda(), b["kv_lens"].cuda(), 32 * words, prefix_len=32)
    complains(ctx)
    fit = 32 * words
    want, places = ref.tree_mask(parents[:fit], batch([fit], [kv - n + fit], 16), words, 32)
    assert torch.equal(mask[:fit].cpu(), want) and torch.equal(positions[:fit].cpu(), places)
    assert bool((mask[fit:] == 0).all()) and bool((positions[fit:] == 32 + kv - n).all())


@pytest.mark.parametrize("n,kv", [(9, 4), (3, 0)])
def test_positions_of_more_nodes_than_keys(ctx, n, kv):
    """The prefix and the depth."""
    b = batch([n], [kv], 16)
    parents = ref.trees([n], seed=2, roots=1)
    mask, positions = g.tree_mask(ctx, parents.cuda(), b["q_start"].cuda(), b["kv_lens"].cuda(), n, prefix_len=48)
    complains(ctx)
    assert positions.tolist() == [48 + len(ref.path(parents, 0, i)) - 1 for i in range(n)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,kv", [([1, 3], [300, 40]), ([5], [5])])
def test_the_largest_group_of_heads(ctx, dtype, d, n_q, kv):
    """128 query heads to a key head: weights and trees."""
    dt, hq, hk, ps = TYPES[dtype], 128, 1, 32
    b = batch(n_q, kv, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    q, scale = normal(sum(n_q), hq, d, seed=3, dtype=dt), 1 / math.sqrt(d)
    mask, _ = ref.tree_mask(ref.trees(n_q), b, 1)
    tree_lse = torch.empty(sum(n_q), hq, device="cuda")
    out = g.tree_attention(ctx, q.cuda(), kd, vd, *on_gpu(b).values(), mask.cuda(), lse=tree_lse)
    lse = attention(q, k, k, b, scale)[1].float()
    weights = torch.rand(b["pages"], hk, ps, generator=torch.Generator().manual_seed(9))
    want, bound = ref.weigh(q, k, b, lse, weights, scale, 2, 0.5)
    got = g.kv_weigh(ctx, q.cuda(), kd, *on_gpu(b).values(), lse.cuda(), weights.cuda(), window=2, decay=0.5).cpu()
    clean(ctx)
    check_attention(out.cpu(), tree_lse.cpu(), *ref.tree_attention(q, k, v, b, mask, scale), (dtype, d, n_q))
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("hk", [129, 200])
def test_many_key_heads(ctx, hk):
    """Weights, choice and moves of more key heads than the short division takes."""
    ps, d, kv, keep = 16, 64, [70, 33, 0], 20
    b = batch([1, 2, 0], kv, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, torch.float16, False)
    q = normal(3, hk, d, seed=3, dtype=torch.float16)
    lse = attention(q, k, k, b, 0.125)[1].float()
    weights = torch.rand(b["pages"], hk, ps, generator=torch.Generator().manual_seed(9))
    want, bound = ref.weigh(q, k, b, lse, weights, 0.125, 0, 1.0)
    at, wd, vd = on_gpu(b), weights.cuda(), kd.clone()
    g.kv_weigh(ctx, q.cuda(), kd, *at.values(), lse.cuda(), wd)
    w = wd.cpu()
    assert bool(((w.double() - want).abs() <= bound).all())
    index, counts = g.kv_select(ctx, wd, at["kv_lens"], at["page_table"], keep, first=1, recent=2)
    g.kv_compact(ctx, kd, vd, at["kv_lens"], at["page_table"], index, counts, weights=wd)
    clean(ctx)
    kept = ref.select(w, kv, b["page_table"], ps, keep, 1, 2)
    assert torch.equal(index.cpu(), kept[0]) and torch.equal(counts.cpu(), kept[1])
    for got, x in zip((kd, vd, wd), ref.compact([k, k, w], b["page_table"], ps, *kept, None)):
        assert torch.equal(got.cpu(), x)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m", [1, 8, 9, 40, 100])
@pytest.mark.parametrize("n", [8, 200])
def test_w4_a_single_group(ctx, dtype, m, n):
    """32 columns: less than a step, and than a copy, of either kernel."""
    a, codes, scales, zeros, bias = w4_inputs(m, n, 32, 32, TYPES[dtype], True)
    y, slack = ref.w4(a, codes, scales, zeros, bias, "none")
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda())
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (dtype, m, n))


def test_a_choice_follows_weights_of_the_call_before(ctx):
    """Weights, choice and moves one after the other without a wait, many times: each reads what the one before wrote."""
    ps, d, hq, hk, kv, keep = 16, 64, 8, 2, [900, 40, 333], 30
    b = batch([1, 1, 1], kv, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, torch.float16, False)
    at, zero = on_gpu(b), torch.zeros(b["pages"], hk, ps, device="cuda")
    wd, runs = zero.clone(), []
    for i in range(40):
        q = normal(3, hq, d, seed=i, dtype=torch.float16)
        lse = attention(q, k, k, b, 0.125)[1].float()
        wd.copy_(zero)
        kk, vv = kd.clone(), kd.clone()
        qd, ld = q.cuda(), lse.cuda()
        torch.cuda.synchronize()
        g.kv_weigh(ctx, qd, kk, *at.values(), ld, wd, decay=0.0)
        index, counts = g.kv_select(ctx, wd, at["kv_lens"], at["page_table"], keep, first=1, recent=2)
        w = wd.clone()
        g.kv_compact(ctx, kk, vv, at["kv_lens"], at["page_table"], index, counts)
        runs.append((w.cpu(), index.cpu(), counts.cpu(), kk.cpu(), vv.cpu()))
    clean(ctx)
    for w, index, counts, kk, vv in runs:
        kept = ref.select(w, kv, b["page_table"], ps, keep, 1, 2)
        assert torch.equal(index, kept[0]) and torch.equal(counts, kept[1])
        want = ref.compact([k, k], b["page_table"], ps, *kept, None)
        assert torch.equal(kk, want[0]) and torch.equal(vv, want[1])
