"""The operators of include/gemm_decode.h on the GPU against their 64-bit definitions."""
import math

import pytest
import torch

import decode_ref as ref
import tensor_core_gemm_tcgen05_gb300 as g
from serving_ref import TYPES, attention, batch, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    with g.Context(0) as c:
        yield c


def clean(ctx):
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_OK, 0)


def complains(ctx):
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_ERR_INDEX, 8)


def normal(*shape, seed, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def cache_of(pages, hk, ps, d, seed, dtype, by_rows):
    """A cache [pages, heads, rows, dim] on the CPU and its copy on the GPU in either order of memory."""
    x = normal(pages, hk, ps, d, seed=seed, dtype=dtype)
    y = x.cuda()
    return x, y.transpose(1, 2).contiguous().transpose(1, 2) if by_rows else y


def on_gpu(b):
    return {k: b[k].cuda() for k in ("q_start", "kv_lens", "page_table")}


# ------------------------------------------------------------------------------------------ trees

@pytest.mark.parametrize("n_q,words", [([1], 1), ([5, 0, 16, 1], 1), ([33, 64, 2], 2), ([0, 0, 40], 3), ([300, 7], 12), ([2048], 64)])
@pytest.mark.parametrize("reach", [1, 9])   # 1: a chain
def test_tree_mask(ctx, n_q, words, reach):
    kv = [n + 11 * i for i, n in enumerate(n_q)]
    b = batch(n_q, kv, 16)
    parents = ref.trees(n_q, seed=3, reach=reach, roots=1 if reach == 1 else 3)
    mask, positions = g.tree_mask(ctx, parents.cuda(), b["q_start"].cuda(), b["kv_lens"].cuda(), 32 * words, prefix_len=48)
    clean(ctx)
    want = ref.tree_mask(parents, b, words, 48)
    assert torch.equal(mask.cpu(), want[0]) and torch.equal(positions.cpu(), want[1])


def test_tree_mask_leaves_padding_alone(ctx):
    n_q = [3, 2]
    b = batch(n_q, [10, 2], 16)
    parents = torch.cat((ref.trees(n_q, roots=1), torch.full((4,), 77, dtype=torch.int32)))
    wide = torch.full((9, 5), -5, dtype=torch.int32, device="cuda")
    positions = torch.full((9,), -5, dtype=torch.int32, device="cuda")
    g.tree_mask(ctx, parents.cuda(), b["q_start"].cuda(), b["kv_lens"].cuda(), 64, mask=wide[:, :2], positions=positions)
    clean(ctx)
    want = ref.tree_mask(parents[:5], b, 2)
    assert torch.equal(wide[:5, :2].cpu(), want[0]) and torch.equal(positions[:5].cpu(), want[1])
    assert bool((wide[5:] == -5).all()) and bool((wide[:, 2:] == -5).all()) and bool((positions[5:] == -5).all())


@pytest.mark.parametrize("parents,words", [([0, 0], 1), ([-2, 0], 1), ([-1, 1], 1), ([-1, 2 ** 30], 1), ([-1] * 40, 1)])
def test_tree_mask_reports_bad_parents(ctx, parents, words):
    n = len(parents)
    b = batch([n], [n + 3], 16)
    mask, positions = g.tree_mask(ctx, torch.tensor(parents, dtype=torch.int32).cuda(), b["q_start"].cuda(), b["kv_lens"].cuda(), 32 * words)
    complains(ctx)
    alone = torch.tensor([[1 << i if i < 31 else -2 ** 31] if i < 32 else [0] for i in range(n)], dtype=torch.int32)
    if n == 2:   # a bad parent counts as none; the second node's good parent stands
        alone[1, 0] = 3 if parents[1] == 0 else 2
    assert torch.equal(mask.cpu(), alone)
    assert int(positions.min()) == 3


TREES = [
    # new tokens, own keys, page size, prefix pages
    ([1], [1], 16, 0),
    ([5], [781], 16, 0),
    ([1, 5, 0, 16, 33], [64, 5, 9, 200, 1033], 16, 0),
    ([16, 3, 9, 12], [400, 70, 9, 1500], 64, 2),
    ([64, 63], [3000, 64], 256, 0),
    ([150, 1], [700, 130], 32, 1),
    ([7] * 20, [40 + 13 * i for i in range(20)], 32, 40),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (2, 2, 64), (14, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree_attention(ctx, dtype, hq, hk, d, case):
    n_q, kv, ps, prefix = TREES[case]
    dt = TYPES[dtype]
    b = batch(n_q, kv, ps, prefix_pages=prefix, seed=case)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, case % 2 == 1)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, case % 2 == 1)
    q = normal(sum(n_q), hq, d, seed=3, dtype=dt)
    parents = ref.trees(n_q, seed=case)
    words = max(1, -(-max(n_q) // 32))
    mask, _ = ref.tree_mask(parents, b, words)
    lse = torch.empty(sum(n_q), hq, device="cuda")
    pre = b["prefix_pages"].cuda() if prefix else None
    out = g.tree_attention(ctx, q.cuda(), kd, vd, *on_gpu(b).values(), mask.cuda(), max_q=max(n_q) if case % 3 else None, prefix_pages=pre, lse=lse)
    clean(ctx)
    check_attention(out.cpu(), lse.cpu(), *ref.tree_attention(q, k, v, b, mask, 1 / math.sqrt(d)), (dtype, hq, hk, d, case))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,ctx_len,words", [(1, 0, 1), (31, 1, 1), (32, 33, 1), (33, 0, 2), (40, 100, 4), (129, 63, 5), (200, 0, 64)])
def test_any_mask(ctx, dtype, n, ctx_len, words):
    """Masks that are no tree: rows that see nothing of the new tokens, not even themselves, and bits past the last."""
    dt = TYPES[dtype]
    hq, hk, d, ps = 4, 2, 64, 16
    b = batch([n, n], [n + ctx_len, n], ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    q = normal(2 * n, hq, d, seed=3, dtype=dt)
    gen = torch.Generator().manual_seed(n)
    mask = torch.randint(0, 2 ** 32, (2 * n, words), generator=gen) & torch.randint(0, 2 ** 32, (2 * n, words), generator=gen)
    mask[:: 3] = 0
    mask[1] = 2 ** 32 - 1
    mask = ref.signed(mask)
    padded = torch.zeros(2 * n, words + 3, dtype=torch.int32)
    padded[:, :words] = mask
    lse = torch.empty(2 * n, hq, device="cuda")
    out = g.tree_attention(ctx, q.cuda(), kd, vd, *on_gpu(b).values(), padded.cuda()[:, :words], lse=lse)
    clean(ctx)
    check_attention(out.cpu(), lse.cpu(), *ref.tree_attention(q, k, v, b, mask, 1 / math.sqrt(d)), (dtype, n, ctx_len, words))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n_q,kv,ps,prefix", [([5, 0, 16], [300, 20, 16], 16, 0), ([16, 3, 9], [400, 70, 9], 64, 2), ([64], [5000], 32, 1),
                                              ([7] * 20, [40 + 13 * i for i in range(20)], 32, 40)])
def test_tree_attention_leaves_padding_alone(ctx, dtype, n_q, kv, ps, prefix):
    """Tokens behind the last sequence are of no sequence, whatever their rows of the mask hold."""
    dt, hq, hk, d, tokens = TYPES[dtype], 8, 2, 128, sum(n_q)
    b = batch(n_q, kv, ps, prefix_pages=prefix, seed=1)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    q = normal(tokens + 37, hq, d, seed=3, dtype=dt)
    q[tokens:] = math.nan
    words = max(1, -(-max(n_q) // 32))
    mask, _ = ref.tree_mask(ref.trees(n_q, seed=2), b, words)
    rows = torch.full((tokens + 37, words), -1, dtype=torch.int32)
    rows[:tokens] = mask
    out = torch.full((tokens + 37, hq, d), 7.0, dtype=dt, device="cuda")
    lse = torch.full((tokens + 37, hq), 7.0, device="cuda")
    g.tree_attention(ctx, q.cuda(), kd, vd, *on_gpu(b).values(), rows.cuda(), prefix_pages=b["prefix_pages"].cuda() if prefix else None,
                     out=out, lse=lse)
    clean(ctx)
    check_attention(out[:tokens].cpu(), lse[:tokens].cpu(), *ref.tree_attention(q[:tokens], k, v, b, mask, 1 / math.sqrt(d)), (dtype, n_q, prefix))
    assert bool((out[tokens:] == 7).all()) and bool((lse[tokens:] == 7).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("n,ctx_len", [(9, 50), (70, 200), (9, 0)])
def test_unseen_nodes_may_hold_anything(ctx, bad, n, ctx_len):
    """The key and value of a node reach the nodes that see it and no others."""
    dt, hq, hk, d, ps = torch.float16, 8, 2, 128, 32
    b = batch([n], [n + ctx_len], ps)
    k, _ = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, _ = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    q = normal(n, hq, d, seed=3, dtype=dt)
    parents = ref.trees([n], seed=5)
    mask, _ = ref.tree_mask(parents, b, 3)
    want = ref.tree_attention(q, k, v, b, mask, 0.1)
    node = 4   # neither first nor last
    place = ctx_len + node
    page, row = int(b["page_table"][0, place // ps]), place % ps
    see = torch.tensor([node in ref.path(parents, 0, i) for i in range(n)])
    assert 0 < int(see.sum()) < n
    for what in ("v", "k"):
        kk, vv = k.clone(), v.clone()
        (vv if what == "v" else kk)[page, :, row] = bad
        lse = torch.empty(n, hq, device="cuda")
        out = g.tree_attention(ctx, q.cuda(), kk.cuda(), vv.cuda(), *on_gpu(b).values(), mask.cuda(), scale=0.1, lse=lse)
        clean(ctx)
        keep = ~see
        check_attention(out.cpu()[keep], lse.cpu()[keep], *(x[keep] for x in want), (bad, n, what))
        if what == "v":
            assert not torch.isfinite(out.cpu()[see].float()).any()


def test_tree_attention_follows_a_replayed_graph(ctx):
    """Lengths, parents and masks that change between the replays of one captured step."""
    dt, hq, hk, d, ps, n = torch.bfloat16, 8, 2, 128, 16, 12
    batches = [batch([n, n], [n + 40, n + 100], ps, width=40, spare=40), batch([n, n], [n + 500, n], ps, width=40, spare=10)]
    pages = max(x["pages"] for x in batches)
    k, kd = cache_of(pages, hk, ps, d, 1, dt, False)
    v, vd = cache_of(pages, hk, ps, d, 2, dt, False)
    q = normal(2 * n, hq, d, seed=3, dtype=dt)
    at = {name: t.clone() for name, t in on_gpu(batches[0]).items()}
    parents = torch.zeros(2 * n, dtype=torch.int32, device="cuda")
    out, lse = torch.empty(2 * n, hq, d, dtype=dt, device="cuda"), torch.empty(2 * n, hq, device="cuda")
    qd = q.cuda()
    at["page_table"].clamp_(max=pages - 1)

    def step():
        mask, _ = g.tree_mask(ctx, parents, at["q_start"], at["kv_lens"], n)
        g.tree_attention(ctx, qd, kd, vd, at["q_start"], at["kv_lens"], at["page_table"], mask, max_q=n, out=out, lse=lse)

    parents.copy_(ref.trees([n, n], seed=0))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, b in enumerate(batches):
        for name, t in on_gpu(b).items():
            at[name].copy_(t)
        p = ref.trees([n, n], seed=10 + i)
        parents.copy_(p)
        graph.replay()
        clean(ctx)
        mask, _ = ref.tree_mask(p, b, 1)
        check_attention(out.cpu(), lse.cpu(), *ref.tree_attention(q, k, v, b, mask, 1 / math.sqrt(d)), i)


@pytest.mark.parametrize("n_q,kv", [([40], [100]), ([8], [5]), ([8], [0])], ids=["past the mask", "more nodes than keys", "no keys"])
def test_tree_attention_reports_what_does_not_fit(ctx, n_q, kv):
    dt, hq, hk, d, ps = torch.float16, 4, 2, 64, 16
    b = batch(n_q, kv, ps)
    _, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    q = normal(n_q[0], hq, d, seed=3, dtype=dt).cuda()
    mask = torch.full((n_q[0], 1), -1, dtype=torch.int32, device="cuda")
    g.tree_attention(ctx, q, kd, kd.clone(), *on_gpu(b).values(), mask)
    complains(ctx)


# --------------------------------------------------------------------------------------- weights

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (2, 2, 64), (14, 2, 64), (40, 2, 128)])
@pytest.mark.parametrize("n_q,kv,ps,window,decay", [
    ([1], [1], 16, 0, 1.0),
    ([1, 1, 0, 1], [300, 17, 40, 256], 16, 0, 1.0),
    ([1, 0, 1], [513, 0, 33], 64, 0, 0.9),
    ([70, 3], [70, 900], 32, 32, 0.0),
    ([20, 33], [20, 290], 1024, 0, 0.5),
    ([5, 9], [3, 8], 16, 0, 1.0),   # more new tokens than keys: the first see none
])
def test_kv_weigh(ctx, dtype, hq, hk, d, n_q, kv, ps, window, decay):
    dt = TYPES[dtype]
    b = batch(n_q, kv, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, ps == 32)
    q = normal(sum(n_q), hq, d, seed=3, dtype=dt)
    scale = 1 / math.sqrt(d)
    lse = attention(q, k, k, b, scale)[1].float()
    gen = torch.Generator().manual_seed(9)
    weights = torch.rand(b["pages"], hk, ps, generator=gen) * 3
    want, bound = ref.weigh(q, k, b, lse, weights, scale, window, decay)
    for s, n in enumerate(n_q):   # what the new tokens' rows held does not matter
        for place in range(max(0, kv[s] - n), kv[s]):
            weights[int(b["page_table"][s, place // ps]), :, place % ps] = math.nan
    got = g.kv_weigh(ctx, q.cuda(), kd, *on_gpu(b).values(), lse.cuda(), weights.cuda(), window=window, decay=decay).cpu()
    clean(ctx)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())


def test_kv_weigh_without_weight(ctx):
    """Tokens whose lse is -inf give nothing, whatever their scores; weights before count as zeros with decay 0."""
    b = batch([2], [40], 16)
    k, kd = cache_of(b["pages"], 1, 16, 64, 1, torch.float16, False)
    q = normal(2, 4, 64, seed=2, dtype=torch.float16)
    q[0, 1] = math.inf
    lse = torch.full((2, 4), -math.inf)
    weights = torch.full((b["pages"], 1, 16), math.nan)
    got = g.kv_weigh(ctx, q.cuda(), kd, *on_gpu(b).values(), lse.cuda(), weights.cuda(), decay=0.0).cpu()
    clean(ctx)
    at = torch.arange(40)
    page = b["page_table"][0].long()[at // 16]
    assert bool((got[page, 0, at % 16] == 0).all())
    got[page, 0, at % 16] = math.nan
    assert bool(got.isnan().all())


def test_kv_weigh_is_the_same_each_time(ctx):
    b = batch([1] * 40, [100 * i + 7 for i in range(40)], 64)
    k, kd = cache_of(b["pages"], 4, 64, 128, 1, torch.bfloat16, False)
    q = normal(40, 16, 128, seed=2, dtype=torch.bfloat16).cuda()
    lse = torch.full((40, 16), 9.0, device="cuda")
    a, c = (g.kv_weigh(ctx, q, kd, *on_gpu(b).values(), lse, torch.ones(b["pages"], 4, 64, device="cuda")) for _ in range(2))
    assert torch.equal(a, c)


def test_more_sequences_than_a_chunk(ctx):
    n_q = [i % 3 for i in range(700)]
    kv = [n + i % 50 for i, n in enumerate(n_q)]
    b = batch(n_q, kv, 16)
    k, kd = cache_of(b["pages"], 1, 16, 64, 1, torch.float16, False)
    q = normal(sum(n_q), 2, 64, seed=3, dtype=torch.float16)
    lse = torch.full((sum(n_q), 2), 3.0)
    weights = torch.rand(b["pages"], 1, 16, generator=torch.Generator().manual_seed(1))
    want, bound = ref.weigh(q, k, b, lse, weights, 0.125, 0, 1.0)
    got = g.kv_weigh(ctx, q.cuda(), kd, *on_gpu(b).values(), lse.cuda(), weights.cuda()).cpu()
    clean(ctx)
    assert bool(((got.double() - want).abs() <= bound).all())


# --------------------------------------------------------------------------------------- eviction

def heavy(pages, hk, ps, seed, kind):
    gen = torch.Generator().manual_seed(seed)
    if kind == "ties":
        return torch.randint(0, 4, (pages, hk, ps), generator=gen).float()
    w = torch.exp(3 * torch.randn(pages, hk, ps, generator=gen))
    if kind == "odd":   # of both signs, zeros of both signs, infinities, NaN
        w *= torch.randint(0, 2, w.shape, generator=gen) * 2 - 1
        u = torch.rand(w.shape, generator=gen)
        for at, x in ((0.1, 0.0), (0.2, -0.0), (0.3, math.inf), (0.4, -math.inf), (0.5, math.nan), (0.6, -math.nan)):
            w = torch.where((u >= at - 0.1) & (u < at), torch.tensor(x), w)
    if kind == "equal":
        w.fill_(0.25)
    return w


@pytest.mark.parametrize("kind", ["plain", "ties", "odd", "equal"])
@pytest.mark.parametrize("kv,ps,keep,first,recent", [
    ([0, 1, 50, 51, 200], 16, 50, 2, 10),
    ([1000, 3], 64, 1, 0, 0),
    ([700, 130], 32, 100, 100, 0),
    ([700, 130], 32, 100, 0, 100),
    ([700, 130], 32, 100, 30, 70),
    ([5000, 9000], 64, 2048, 4, 512),
    ([40], 16, 0, 0, 0),
    ([40, 41], 1024, 40, 1, 1),
])
def test_kv_select(ctx, kind, kv, ps, keep, first, recent):
    b = batch([0] * len(kv), kv, ps)
    w = heavy(b["pages"], 3, ps, 4, kind)
    index, counts = g.kv_select(ctx, w.cuda(), b["kv_lens"].cuda(), b["page_table"].cuda(), keep, first=first, recent=recent)
    clean(ctx)
    want = ref.select(w, kv, b["page_table"], ps, keep, first, recent)
    assert torch.equal(counts.cpu(), want[1])
    assert torch.equal(index.cpu(), want[0])


@pytest.mark.parametrize("kv,heads", [(100_000, 1), (450_000, 1), (60_000, 300)])
def test_kv_select_long(ctx, kv, heads):
    """Lists that a cluster shares, one past what its CTAs hold, and one past that of a single CTA (300 heads)."""
    ps, keep = 1024, 30_000
    b = batch([0], [kv], ps)
    w = heavy(b["pages"], heads, ps, 4, "plain")
    index, counts = g.kv_select(ctx, w.cuda(), b["kv_lens"].cuda(), b["page_table"].cuda(), keep, first=4, recent=100)
    clean(ctx)
    assert counts.tolist() == [keep]
    at = torch.arange(kv)
    for h in {0, heads // 2, heads - 1}:
        x = w[b["page_table"][0].long()[at // ps], h, at % ps]
        x[:4] = math.inf
        x[-100:] = math.inf
        want = torch.sort(x, descending=True, stable=True).indices[:keep].sort().values
        assert torch.equal(index[0, h].cpu().long(), want)


def test_kv_select_strides(ctx):
    kv, ps = [300, 20, 90], 16
    b = batch([0] * 3, kv, ps)
    w = heavy(b["pages"], 2, ps, 4, "plain")
    wide = torch.full((b["pages"], 4, ps + 5), math.nan, device="cuda")
    wide[:, ::2, :ps] = w.cuda()
    index = torch.full((3, 4, 70), -7, dtype=torch.int32, device="cuda")
    _, counts = g.kv_select(ctx, wide[:, ::2, :ps], b["kv_lens"].cuda(), b["page_table"].cuda(), 64, first=1, recent=5, index=index[:, ::2, :64])
    clean(ctx)
    want = ref.select(w, kv, b["page_table"], ps, 64, 1, 5)
    assert torch.equal(index[:, ::2, :64].cpu(), want[0]) and torch.equal(counts.cpu(), want[1])
    assert bool((index[:, 1::2] == -7).all()) and bool((index[:, :, 64:] == -7).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d,hk,ps,by_rows", [(128, 3, 16, False), (64, 2, 64, True), (128, 1, 1024, True), (64, 8, 32, False)])
@pytest.mark.parametrize("kv,keep", [([60, 5, 0, 33], 20), ([5000], 2500), ([900, 3000], 700), ([40], 40)])
def test_kv_compact(ctx, dtype, d, hk, ps, by_rows, kv, keep):
    """A list for each head, and the weights moved along."""
    dt = TYPES[dtype]
    b = batch([0] * len(kv), kv, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, by_rows)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, by_rows)
    w = heavy(b["pages"], hk, ps, 3, "plain")
    wd = w.cuda()
    index, counts = ref.select(w, kv, b["page_table"], ps, keep, 2, 3)
    lens = g.kv_compact(ctx, kd, vd, b["kv_lens"].cuda(), b["page_table"].cuda(), index.cuda(), counts.cuda(), weights=wd)
    clean(ctx)
    want = ref.compact([k, v, w], b["page_table"], ps, index, counts, None)
    assert torch.equal(lens.cpu(), counts)
    for got, x in zip((kd, vd, wd), want):
        assert torch.equal(got.cpu(), x)


@pytest.mark.parametrize("d,hk,most", [(128, 8, 4), (64, 16, 12), (128, 2, 70), (64, 1, 1)])
def test_kv_compact_takes_over_a_path(ctx, d, hk, most):
    """One list for all heads, behind a text of each sequence's own."""
    ps, dt = 16, torch.bfloat16
    n_q = [1, 30, 0, 80, 17]
    kv = [n + 37 * i for i, n in enumerate(n_q)]
    b = batch(n_q, kv, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, True)
    kd = kd.transpose(1, 2).contiguous().transpose(1, 2)
    gen = torch.Generator().manual_seed(most)
    index, counts = torch.full((5, most), -3, dtype=torch.int32), []
    for s, n in enumerate(n_q):
        path = torch.randperm(n, generator=gen)[:most].sort().values if n else torch.zeros(0)
        index[s, : len(path)] = path
        counts.append(len(path))
    counts = torch.tensor(counts, dtype=torch.int32)
    start = b["kv_lens"] - torch.tensor(n_q, dtype=torch.int32)
    lens = g.kv_compact(ctx, kd, vd, b["kv_lens"].cuda(), b["page_table"].cuda(), index.cuda(), counts.cuda(), start=start.cuda())
    clean(ctx)
    want = ref.compact([k, v], b["page_table"], ps, index, counts, start)
    assert torch.equal(lens.cpu(), start + counts)
    assert torch.equal(kd.cpu(), want[0]) and torch.equal(vd.cpu(), want[1])


@pytest.mark.parametrize("what", ["descending", "past the end", "count", "start", "page"])
def test_kv_compact_reports_what_it_does_not_move(ctx, what):
    ps, hk, d = 16, 2, 64
    b = batch([0, 0], [40, 40], ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, torch.float16, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, torch.float16, False)
    index = torch.tensor([[0, 5, 9], [2, 20, 39]], dtype=torch.int32)
    counts, start, table = torch.tensor([3, 3], dtype=torch.int32), torch.zeros(2, dtype=torch.int32), b["page_table"].clone()
    good = index.clone()
    lens = [3, 3]
    if what == "descending":
        index[1] = torch.tensor([2, 0, 39])
        good[1] = torch.tensor([2, 1, 39])   # (entry 1 stays where it is)
    elif what == "past the end":
        index[1, 2] = 40
        good[1, 2] = 2
    elif what == "count":
        counts[0] = 4
        counts[1] = -1
        lens = [3, 0]
    elif what == "start":
        start[0], start[1] = -1, 41
        lens = [0, 40]
    else:
        table[1, 2] = b["pages"]
        good[1, 2] = 2
    got = g.kv_compact(ctx, kd, vd, b["kv_lens"].cuda(), table.cuda(), index.cuda(), counts.cuda(), start=start.cuda())
    complains(ctx)
    moved = {"count": [3, 0], "start": [0, 0]}.get(what, [3, 3])
    want = ref.compact([k, v], b["page_table"], ps, good, torch.tensor(moved), None)
    assert got.tolist() == lens
    assert torch.equal(kd.cpu(), want[0]) and torch.equal(vd.cpu(), want[1])


# ------------------------------------------------------------------------------------------- 4 bits

def w4_inputs(m, n, k, group, dt, zeros, seed=0):
    gen = torch.Generator().manual_seed(seed)
    a = torch.randn(m, k, generator=gen).to(dt)
    codes = torch.randint(0, 256, (n, k // 2), generator=gen, dtype=torch.uint8)
    scales = ((torch.rand(n, k // group, generator=gen) + 0.5) * torch.where(torch.rand(n, k // group, generator=gen) < 0.2, -0.1, 0.1)).to(dt)
    z = torch.randint(0, 256, (n, k // group), generator=gen, dtype=torch.uint8) if zeros else None   # (the high bits do not count)
    bias = torch.randn(n, generator=gen).to(dt)
    return a, codes, scales, z, bias


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,groups", [(1, 8, 1), (1, 136, 5), (3, 2048, 8), (8, 256, 17), (9, 128, 4), (16, 1000, 9), (17, 264, 3),
                                        (33, 136, 12), (64, 640, 7), (65, 128, 4), (130, 24, 2)])
def test_w4(ctx, dtype, group, m, n, groups):
    dt = TYPES[dtype]
    a, codes, scales, zeros, bias = w4_inputs(m, n, group * groups, group, dt, zeros=(m + groups) % 2 == 0)
    act = ["none", "gelu", "relu"][(m + n // 8 + groups) % 3]
    y, slack = ref.w4(a, codes, scales, zeros, bias if m % 2 else None, act)
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), None if zeros is None else zeros.cuda(), bias.cuda() if m % 2 else None,
                    {"none": g.EPI_NONE, "gelu": g.EPI_GELU, "relu": g.EPI_RELU}[act])
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (dtype, group, m, n, groups, act))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (8, 16384, 1024), (64, 1024, 8192), (24, 96, 16384)])
def test_w4_large(ctx, dtype, m, n, k):
    dt = TYPES[dtype]
    a, codes, scales, zeros, bias = w4_inputs(m, n, k, 128, dt, True)
    y, slack = ref.w4(a, codes, scales, zeros, bias, "none")
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda())
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (dtype, m, n, k))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k,group", [(1, 4096, 16384, 64), (3, 8192, 4096, 128), (5, 4096, 8192, 128), (8, 2048, 16384, 32),
                                           (1, 24, 65536, 32), (2, 16, 69632, 128), (2, 16, 69888, 128), (8, 8, 131072, 64), (4, 50000, 256, 128)])
def test_w4_few_rows(ctx, dtype, m, n, k, group):
    """Where the faster kernel for up to eight rows depends on the sizes, the group and the type."""
    dt = TYPES[dtype]
    a, codes, scales, zeros, bias = w4_inputs(m, n, k, group, dt, True, seed=m)
    y, slack = ref.w4(a, codes, scales, zeros, bias, "relu")
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda(), g.EPI_RELU)
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (dtype, m, n, k, group))


def test_w4_rows_of_any_stride(ctx):
    a, codes, scales, zeros, bias = w4_inputs(5, 64, 256, 64, torch.float16, True)
    wide = torch.full((5, 300 + 4), 7.0, dtype=torch.float16, device="cuda")
    wide[:, :256] = a.cuda()
    out = torch.full((5, 80), -7.0, dtype=torch.float16, device="cuda")
    g.w4_gemm(ctx, wide[:, :256], codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda(), out=out[:, :64])
    clean(ctx)
    y, slack = ref.w4(a, codes, scales, zeros, bias, "none")
    ref.check_w4(out[:, :64].cpu(), y, slack, "strides")
    assert bool((out[:, 64:] == -7).all())


@pytest.mark.parametrize("act", ["none", "gelu", "relu"])
def test_w4_without_columns(ctx, act):
    bias = torch.tensor([-2.0, 0.5, 3.0, -0.1] * 4, dtype=torch.bfloat16)
    a, codes, scales = torch.empty(3, 0, dtype=torch.bfloat16), torch.empty(16, 0, dtype=torch.uint8), torch.empty(16, 0, dtype=torch.bfloat16)
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), None, bias.cuda(), {"none": g.EPI_NONE, "gelu": g.EPI_GELU, "relu": g.EPI_RELU}[act])
    clean(ctx)
    y, slack = ref.w4(a, codes, scales, None, bias, act)
    ref.check_w4(got.cpu(), y.expand(3, 16), slack, act)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m", [2, 40])
@pytest.mark.parametrize("act", ["none", "gelu", "relu"])
def test_w4_numbers_that_are_not_finite(ctx, dtype, m, act):
    """They stay in their row of A, and NaN stays NaN through the activations."""
    dt = TYPES[dtype]
    a, codes, scales, zeros, _ = w4_inputs(m, 64, 256, 32, dt, True)
    y, slack = ref.w4(a, codes, scales, zeros, None, act)
    a[1, 100] = math.nan
    epi = {"none": g.EPI_NONE, "gelu": g.EPI_GELU, "relu": g.EPI_RELU}[act]
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), epilogue=epi).cpu()
    clean(ctx)
    assert bool(got[1].isnan().all())
    keep = torch.arange(m) != 1
    ref.check_w4(got[keep], y[keep], slack[keep], (dtype, m, act))
    # of A's infinities, those whose code is the zero give NaN, the others an infinity of the weight's sign
    a[1] = 0
    a[1, 100] = math.inf
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), epilogue=epi).cpu()[1].float()
    w = ((codes[:, 50] % 16).float() - (zeros[:, 3] % 16).float()) * scales[:, 3].float()
    want = w * math.inf
    want = torch.where(want < 0, torch.zeros(()), want) if act != "none" else want
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])
