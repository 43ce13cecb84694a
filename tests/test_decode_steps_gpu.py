"""The operators of include/gemm_decode.h together, as a serving loop uses them, and the calls a loop makes of them out of
the ordinary: captured, on other streams, over caches whose offsets pass 32 bits, refused."""
import math

import pytest
import torch

import decode_ref as ref
import serving_ref
import tensor_core_gemm_tcgen05_gb300 as g
from serving_ref import attention, batch, check_attention, check_rope
from test_decode_gpu import cache_of, clean, heavy, normal, on_gpu, w4_inputs

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module")
def ctx():
    with g.Context(0) as c:
        yield c


def test_drafts_verified_and_taken_over(ctx):
    """Masks and positions from the parents, rotation, append, tree attention, the deepest path taken over; then a plain
    decoding step on the cache that this leaves."""
    hq, hk, d, ps, dt = 8, 2, 64, 16, F16
    texts, n_q = [5, 40, 17, 0], [7, 1, 12, 3]
    b = batch(n_q, [t + n for t, n in zip(texts, n_q)], ps, width=6, spare=8)
    for s in range(4):   # (room for the next step's tokens)
        b["page_table"][s, -(-b["kv"][s] // ps) :] = 0
        if b["kv"][s] % ps == 0:
            b["page_table"][s, b["kv"][s] // ps] = b["pages"] - 1 - s
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    tokens = sum(n_q)
    q, k_new, v_new = normal(tokens, hq, d, seed=3, dtype=dt), normal(tokens, hk, d, seed=4, dtype=dt), normal(tokens, hk, d, seed=5, dtype=dt)
    parents = ref.trees(n_q, seed=6, roots=1)
    table, _ = g.rope_table(d)
    at = on_gpu(b)
    mask, positions = g.tree_mask(ctx, parents.cuda(), at["q_start"], at["kv_lens"], max(n_q))
    q2, k2 = g.qk_rope(ctx, q.cuda(), k_new.cuda(), positions, table.cuda())
    g.kv_append(ctx, None, k2, v_new.cuda(), kd, vd, *at.values())
    lse = torch.empty(tokens, hq, device="cuda")
    out = g.tree_attention(ctx, q2, kd, vd, *at.values(), mask, max_q=max(n_q), lse=lse)
    clean(ctx)
    want_mask, want_positions = ref.tree_mask(parents, b, 1)
    assert torch.equal(mask.cpu(), want_mask) and torch.equal(positions.cpu(), want_positions)
    check_rope(q2.cpu(), *serving_ref.rope(q, None, want_positions.tolist(), table, False, 1.0, 0), "q")
    check_rope(k2.cpu(), *serving_ref.rope(k_new, None, want_positions.tolist(), table, False, 1.0, 0), "k")
    q2, k2 = q2.cpu(), k2.cpu()
    for s, n in enumerate(n_q):
        for i in range(n):
            row, t = texts[s] + i, int(b["q_start"][s]) + i
            k[b["page_table"][s, row // ps], :, row % ps], v[b["page_table"][s, row // ps], :, row % ps] = k2[t], v_new[t]
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)
    check_attention(out.cpu(), lse.cpu(), *ref.tree_attention(q2, k, v, b, want_mask, 1 / math.sqrt(d)), "tree")
    # the deepest node's path
    index, counts = torch.zeros(4, 12, dtype=torch.int32), []
    for s, n in enumerate(n_q):
        a = int(b["q_start"][s])
        deepest = max(range(n), key=lambda i: len(ref.path(parents, a, i)))
        line = ref.path(parents, a, deepest)[::-1]
        index[s, : len(line)] = torch.tensor(line)
        counts.append(len(line))
    counts, start = torch.tensor(counts, dtype=torch.int32), torch.tensor(texts, dtype=torch.int32)
    lens = g.kv_compact(ctx, kd, vd, at["kv_lens"], at["page_table"], index.cuda(), counts.cuda(), start=start.cuda())
    assert lens.tolist() == (start + counts).tolist()
    for s in range(4):   # the rows of the accepted tokens, in the order of their positions
        for j in range(int(counts[s])):
            t, row = int(b["q_start"][s]) + int(index[s, j]), texts[s] + j
            assert int(want_positions[t]) == row
            k[b["page_table"][s, row // ps], :, row % ps], v[b["page_table"][s, row // ps], :, row % ps] = k2[t], v_new[t]
    # one more token each
    q, k_new, v_new = (normal(4, h, d, seed=7 + i, dtype=dt) for i, h in enumerate((hq, hk, hk)))
    q_start, kv_lens = torch.arange(5, dtype=torch.int32, device="cuda"), lens + 1
    q2 = g.kv_append(ctx, q.cuda(), k_new.cuda(), v_new.cuda(), kd, vd, q_start, kv_lens, at["page_table"], table.cuda())
    lse = torch.empty(4, hq, device="cuda")
    out = g.paged_attention(ctx, q2, kd, vd, q_start, kv_lens, at["page_table"], max_q=1, lse=lse)
    clean(ctx)
    k3 = serving_ref.rope(k_new, None, lens.tolist(), table, False, 1.0, 0)[0].to(dt)
    now = dict(b, n_q=[1] * 4, kv=kv_lens.tolist(), q_start=q_start.cpu(), kv_lens=kv_lens.cpu())
    for s, row in enumerate(lens.tolist()):
        got = kd[b["page_table"][s, row // ps], :, row % ps].cpu()
        assert float((got.double() - k3[s].double()).abs().max()) < 2e-2   # (checked as such elsewhere: the row is the right one)
        k[b["page_table"][s, row // ps], :, row % ps], v[b["page_table"][s, row // ps], :, row % ps] = got, v_new[s]
    check_attention(out.cpu(), lse.cpu(), *attention(q2.cpu(), k, v, now, 1 / math.sqrt(d)), "next")


@pytest.mark.parametrize("captured", [False, True])
def test_a_cache_kept_to_its_size(ctx, captured):
    """Decoding steps that add up attention weight, evictions in between; the same captured into one graph and replayed."""
    hq, hk, d, ps, dt, keep = 4, 2, 128, 16, torch.bfloat16, 40
    seqs, lens0, width = 3, [39, 70, 12], 8
    b = batch([1] * seqs, [width * ps - 1] * seqs, ps)
    k, kd = cache_of(b["pages"], hk, ps, d, 1, dt, False)
    v, vd = cache_of(b["pages"], hk, ps, d, 2, dt, False)
    weights = torch.rand(b["pages"], hk, ps, generator=torch.Generator().manual_seed(3))
    wd = weights.cuda()
    q_start, table, page_table = b["q_start"].cuda(), g.rope_table(d)[0].cuda(), b["page_table"].cuda()
    kv = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    q, k_new, v_new = (torch.zeros(seqs, h, d, dtype=dt, device="cuda") for h in (hq, hk, hk))
    position = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    lse, out = torch.empty(seqs, hq, device="cuda"), torch.empty(seqs, hq, d, dtype=dt, device="cuda")
    q2, k2 = torch.empty_like(q), torch.empty_like(k_new)
    index, counts = torch.empty(seqs, hk, keep, dtype=torch.int32, device="cuda"), torch.empty(seqs, dtype=torch.int32, device="cuda")
    before, kept = torch.empty_like(wd), torch.empty_like(kv)

    def step():
        kv.add_(1)
        g.qk_rope(ctx, q, k_new, position, table, q_out=q2, k_out=k2)
        position.add_(1)
        g.kv_append(ctx, None, k2, v_new, kd, vd, q_start, kv, page_table)
        g.paged_attention(ctx, q2, kd, vd, q_start, kv, page_table, max_q=1, out=out, lse=lse)
        g.kv_weigh(ctx, q2, kd, q_start, kv, page_table, lse, wd, decay=0.75)
        before.copy_(wd)
        g.kv_select(ctx, wd, kv, page_table, keep, first=1, recent=8, index=index, counts=counts)
        g.kv_compact(ctx, kd, vd, kv, page_table, index, counts, weights=wd, new_lens=kept)
        kv.copy_(kept)

    graph = None
    state = [kd, vd, wd, kv, position]
    if captured:
        saved = [x.clone() for x in state]
        step()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step()
        for x, y in zip(state, saved):
            x.copy_(y)
    lens = list(lens0)
    for i in range(4):
        for j, (t, h) in enumerate(((q, hq), (k_new, hk), (v_new, hk))):
            t.copy_(normal(seqs, h, d, seed=100 * i + j, dtype=dt))
        graph.replay() if captured else step()
        clean(ctx)
        lens = [n + 1 for n in lens]
        now = dict(b, kv=lens, kv_lens=torch.tensor(lens, dtype=torch.int32))
        for s, n in enumerate(lens):
            at = (b["page_table"][s, (n - 1) // ps], slice(None), (n - 1) % ps)
            k[at], v[at] = k2[s].cpu(), v_new[s].cpu()
        scale = 1 / math.sqrt(d)
        check_attention(out.cpu(), lse.cpu(), *attention(q2.cpu(), k, v, now, scale), i)
        want, bound = ref.weigh(q2.cpu(), k, now, lse.cpu(), weights, scale, 0, 0.75)
        weights = before.cpu()
        assert bool(((weights.double() - want).abs() <= bound).all())
        kept_index, kept_counts = ref.select(weights, lens, b["page_table"], ps, keep, 1, 8)
        assert torch.equal(index.cpu(), kept_index) and torch.equal(counts.cpu(), kept_counts)
        k, v, weights = ref.compact([k, v, weights], b["page_table"], ps, kept_index, kept_counts, None)
        lens = kept_counts.tolist()
        assert kv.tolist() == lens
        for got, x in zip((kd, vd, wd), (k, v, weights)):
            assert torch.equal(got.cpu(), x)


@pytest.mark.parametrize("m", [3, 40])
def test_w4_captured_with_new_inputs(ctx, m):
    a, codes, scales, zeros, bias = w4_inputs(m, 264, 512, 64, F16, True)
    ad = torch.zeros_like(a).cuda()
    dev = [x.cuda() for x in (codes, scales, zeros, bias)]
    out = torch.empty(m, 264, dtype=F16, device="cuda")

    def run():
        g.w4_gemm(ctx, ad, dev[0], dev[1], dev[2], dev[3], g.EPI_GELU, out=out)

    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for seed in (1, 2):
        a, codes, scales, zeros, bias = w4_inputs(m, 264, 512, 64, F16, True, seed=seed)
        ad.copy_(a)
        for x, y in zip(dev, (codes, scales, zeros, bias)):
            x.copy_(y)
        graph.replay()
        clean(ctx)
        ref.check_w4(out.cpu(), *ref.w4(a, codes, scales, zeros, bias, "gelu"), seed)


def test_on_another_stream(ctx):
    """Calls queued on a stream of their own, what they return used there; the current stream is busy meanwhile."""
    b = batch([4, 9], [300, 70], 16)
    hq, hk, d = 8, 2, 64
    k, kd = cache_of(b["pages"], hk, 16, d, 1, F16, False)
    v, vd = cache_of(b["pages"], hk, 16, d, 2, F16, False)
    q = normal(13, hq, d, seed=3, dtype=F16)
    parents = ref.trees([4, 9])
    w = heavy(b["pages"], hk, 16, 4, "plain")
    a, codes, scales, zeros, _ = w4_inputs(20, 128, 256, 128, F16, True)
    at, qd, pd, wd = on_gpu(b), q.cuda(), parents.cuda(), w.cuda()
    w4 = [x.cuda() for x in (a, codes, scales, zeros)]
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    mask, _ = g.tree_mask(ctx, pd, at["q_start"], at["kv_lens"], 9, stream=side)
    out = g.tree_attention(ctx, qd, kd, vd, *at.values(), mask, stream=side)
    index, counts = g.kv_select(ctx, wd, at["kv_lens"], at["page_table"], 50, stream=side)
    lens = g.kv_compact(ctx, kd, vd, at["kv_lens"], at["page_table"], index, counts, stream=side)
    y = g.w4_gemm(ctx, *w4, stream=side)
    side.synchronize()
    want = ref.tree_mask(parents, b, 1)[0]
    assert torch.equal(mask.cpu(), want)
    o, _, spread = ref.tree_attention(q, k, v, b, want, 1 / math.sqrt(d))
    assert float(((out.cpu().double() - o).abs() / (2.0 ** -10 * (spread + o.abs()) + 1e-6)).max()) <= 1
    kept = ref.select(w, b["kv"], b["page_table"], 16, 50, 0, 0)
    assert torch.equal(index.cpu(), kept[0]) and torch.equal(counts.cpu(), kept[1]) and torch.equal(lens.cpu(), kept[1])
    moved = ref.compact([k, v], b["page_table"], 16, *kept, None)
    assert torch.equal(kd.cpu(), moved[0]) and torch.equal(vd.cpu(), moved[1])
    ref.check_w4(y.cpu(), *ref.w4(a, codes, scales, zeros, None, "none"), "side")
    clean(ctx)


def test_offsets_past_32_bits(ctx):
    """Caches and weights whose pages lie more than 2^31 elements apart."""
    hq, hk, d, ps, pages, stride = 4, 2, 64, 16, 4, 2 ** 31 + 64
    wide = torch.empty(3 * stride + hk * ps, dtype=torch.float32, device="cuda")
    big = torch.empty(3 * stride + 2 * hk * ps * d, dtype=F16, device="cuda")
    kd = big.as_strided((pages, hk, ps, d), (stride, ps * d, d, 1))
    vd = big.as_strided((pages, hk, ps, d), (stride, ps * d, d, 1), hk * ps * d)
    wd = wide.as_strided((pages, hk, ps), (stride, ps, 1))
    b = batch([5], [60], ps, spare=0)
    b["page_table"] = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32)
    k, v, q = normal(pages, hk, ps, d, seed=1, dtype=F16), normal(pages, hk, ps, d, seed=2, dtype=F16), normal(5, hq, d, seed=3, dtype=F16)
    w = heavy(pages, hk, ps, 4, "plain")
    kd.copy_(k), vd.copy_(v), wd.copy_(w)
    parents = ref.trees([5])
    at = on_gpu(b)
    mask, _ = g.tree_mask(ctx, parents.cuda(), at["q_start"], at["kv_lens"], 5)
    lse = torch.empty(5, hq, device="cuda")
    out = g.tree_attention(ctx, q.cuda(), kd, vd, *at.values(), mask, lse=lse)
    clean(ctx)
    check_attention(out.cpu(), lse.cpu(), *ref.tree_attention(q, k, v, b, mask.cpu(), 1 / math.sqrt(d)), "far")
    full = attention(q, k, v, b, 1 / math.sqrt(d))[1].float()
    want, bound = ref.weigh(q, k, b, full, w, 1 / math.sqrt(d), 0, 1.0)
    g.kv_weigh(ctx, q.cuda(), kd, *at.values(), full.cuda(), wd)
    clean(ctx)
    assert bool(((wd.cpu().double() - want).abs() <= bound).all())
    w = wd.cpu()
    kept = ref.select(w, [60], b["page_table"], ps, 20, 1, 2)
    index, counts = g.kv_select(ctx, wd, at["kv_lens"], at["page_table"], 20, first=1, recent=2)
    g.kv_compact(ctx, kd, vd, at["kv_lens"], at["page_table"], index, counts, weights=wd)
    clean(ctx)
    assert torch.equal(index.cpu(), kept[0])
    for got, x in zip((kd, vd, wd), ref.compact([k, v, w], b["page_table"], ps, *kept, None)):
        assert torch.equal(got.cpu(), x)


@pytest.mark.parametrize("m", [1, 20])
def test_w4_codes_past_32_bits(ctx, m):
    """More than 2^32 bytes of codes; the last rows are looked at."""
    n, k, group = 2 ** 16 + 16, 2 ** 17 + 128, 128
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, k // group), 0.01, dtype=F16, device="cuda")
    a, c, s, _, _ = w4_inputs(m, 24, k, group, F16, False)
    codes[-24:], scales[-24:] = c.cuda(), s.cuda()
    got = g.w4_gemm(ctx, a.cuda(), codes, scales)
    clean(ctx)
    ref.check_w4(got[:, -24:].cpu(), *ref.w4(a, c, s, None, None, "none"), m)


@pytest.mark.parametrize("what", ["w4", "tree"])
def test_a_wait_that_runs_out_is_reported(ctx, what):
    """An operand that never arrives (held back by the test hook); the next call is as always."""
    a, codes, scales, zeros, _ = w4_inputs(20, 128, 512, 128, F16, True)
    b = batch([3], [40], 16)
    k, kd = cache_of(b["pages"], 1, 16, 64, 1, F16, False)
    q, parents = normal(3, 2, 64, seed=2, dtype=F16), ref.trees([3])
    mask = ref.tree_mask(parents, b, 1)[0]
    vd = kd.clone()

    def call():
        if what == "w4":
            return g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda())
        return g.tree_attention(ctx, q.cuda(), kd, vd, *on_gpu(b).values(), mask.cuda())

    g.gemm_set_timeout_ns(ctx, 2_000_000)
    g.gemm_set_debug(ctx, g.GEMM_DEBUG_WITHHOLD_FIRST_LOAD)
    try:
        call()
        torch.cuda.synchronize()
        assert g.gemm_last_device_error(ctx)[0] == g.GEMM_ERR_TIMEOUT
    finally:
        g.gemm_set_debug(ctx, 0)
        g.gemm_set_timeout_ns(ctx, 2_000_000_000)
    got = call()
    clean(ctx)
    if what == "w4":
        ref.check_w4(got.cpu(), *ref.w4(a, codes, scales, zeros, None, "none"), "after")
    else:
        o = ref.tree_attention(q, k, k, b, mask, 1 / 8)[0]
        assert float((got.cpu().double() - o).abs().max()) < 1e-2


# ----------------------------------------------------------------------------------------- refusals

def status(call):
    with pytest.raises(g.GemmError) as e:
        call()
    return e.value.status


def test_refusals(ctx):
    """What the library refuses before anything is enqueued."""
    hk, d, ps = 2, 64, 16
    b = batch([3], [40], ps)
    _, kd = cache_of(b["pages"], hk, ps, d, 1, F16, False)
    vd, at = kd.clone(), on_gpu(b)
    q = torch.zeros(3, 4, d, dtype=F16, device="cuda")
    mask, lse = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, device="cuda")
    w = torch.zeros(b["pages"], hk, ps, device="cuda")
    ARG, ALIGN, DEVICE = g.GEMM_ERR_ARG, g.GEMM_ERR_ALIGN, g.GEMM_ERR_DEVICE

    def tree(mask=mask, q=q, **kw):
        return g.tree_attention(ctx, q, kd, vd, *at.values(), mask, **kw)

    assert status(lambda: tree(torch.zeros(3, 65, dtype=torch.int32, device="cuda"))) == ARG
    assert status(lambda: tree(torch.zeros(3, 0, dtype=torch.int32, device="cuda"))) == ARG
    assert status(lambda: tree(out=q)) == ARG
    assert status(lambda: tree(q=q[:, :3])) == ARG
    assert status(lambda: tree(scale=math.inf)) == ARG
    assert status(lambda: tree(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))) == ARG
    over = torch.zeros(3, 4, d, dtype=F16, device="cuda")
    assert status(lambda: tree(over.view(torch.int32).flatten()[:3].view(3, 1), out=over)) == ARG
    parents = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert status(lambda: g.tree_mask(ctx, parents, at["q_start"], at["kv_lens"], 3, prefix_len=-1)) == ARG
    assert status(lambda: g.tree_mask(ctx, parents, at["q_start"], at["kv_lens"], 3, positions=parents)) == ARG
    assert status(lambda: g.tree_mask(ctx, parents, at["q_start"], at["kv_lens"], 3, mask=torch.zeros(3, 65, dtype=torch.int32, device="cuda"))) == ARG

    def weigh(q=q, cache=kd, lse=lse, w=w, **kw):
        return g.kv_weigh(ctx, q, cache, *at.values(), lse, w, **kw)

    for kw in (dict(decay=-0.5), dict(decay=1.5), dict(decay=math.nan), dict(window=-1), dict(scale=math.nan), dict(q=q[:, :3], lse=lse[:, :3]),
               dict(lse=w.flatten()[:12].view(3, 4)), dict(w=w[:, :1].expand(-1, hk, -1))):
        assert status(lambda: weigh(**kw)) == ARG, kw

    def select(keep=8, w=w, **kw):
        return g.kv_select(ctx, w, at["kv_lens"], at["page_table"], keep, **kw)

    for kw in (dict(first=9), dict(recent=9), dict(first=5, recent=4), dict(first=-1), dict(recent=-1), dict(w=torch.zeros(5, hk, 24, device="cuda")),
               dict(index=torch.zeros(1, 1, 8, dtype=torch.int32, device="cuda").expand(1, hk, 8)), dict(counts=at["kv_lens"])):
        assert status(lambda: select(**kw)) == ARG, kw
    index, counts = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")

    def compact(k=kd, v=vd, index=index, counts=counts, **kw):
        return g.kv_compact(ctx, k, v, at["kv_lens"], at["page_table"], index, counts, **kw)

    for kw in (dict(v=kd), dict(new_lens=at["kv_lens"]), dict(new_lens=counts), dict(start=counts, new_lens=counts),
               dict(index=kd.view(torch.int32).flatten()[:4].view(1, 4)), dict(weights=w, new_lens=w.view(torch.int32).flatten()[:1])):
        assert status(lambda: compact(**kw)) == ARG, kw
    a, codes, scales, zeros, bias = (x.cuda() for x in w4_inputs(2, 16, 128, 64, F16, True))

    def w4(a=a, codes=codes, scales=scales, zeros=zeros, **kw):
        return g.w4_gemm(ctx, a, codes, scales, zeros, **kw)

    assert status(lambda: w4(epilogue=g.EPI_SOFTMAX)) == ARG
    assert status(lambda: w4(epilogue=7)) == ARG
    assert status(lambda: w4(codes=codes[:12].contiguous(), scales=scales[:12].contiguous(), zeros=zeros[:12].contiguous())) == ALIGN
    assert status(lambda: w4(scales=scales[:, :1].repeat(1, 8).contiguous(), zeros=None)) == ARG   # groups of 16
    big = torch.zeros(2, 132, dtype=F16, device="cuda")
    assert status(lambda: w4(a=big[:, :128])) == ALIGN
    assert status(lambda: w4(a=torch.zeros(264, dtype=F16, device="cuda")[4:260].view(2, 128))) == ALIGN
    assert status(lambda: w4(out=a[:, :16])) == ARG
    assert status(lambda: w4(bias=torch.zeros(24, dtype=F16, device="cuda")[1:17])) == ALIGN
    # memory of the host
    assert status(lambda: g.w4_gemm(ctx, *(x.cpu() for x in (a, codes, scales, zeros)), stream=0)) == DEVICE
    host = [x.cpu() for x in (kd, vd, at["kv_lens"], at["page_table"], index, counts)]
    assert status(lambda: g.kv_compact(ctx, *host, stream=0)) == DEVICE
    assert status(lambda: g.kv_select(ctx, w.cpu(), host[2], host[3], 4, stream=0)) == DEVICE
    clean(ctx)


def test_nothing_to_do(ctx):
    """No tokens, no sequences, nothing to keep."""
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    _, kd = cache_of(3, 2, 16, 64, 1, F16, False)
    vd, w = kd.clone(), torch.ones(3, 2, 16, device="cuda")
    q_start, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    q, lse = torch.zeros(0, 4, 64, dtype=F16, device="cuda"), torch.zeros(0, 4, device="cuda")
    mask, positions = g.tree_mask(ctx, none, q_start, none, 0)
    assert mask.shape == (0, 1) and positions.shape == (0,)
    assert g.tree_attention(ctx, q, kd, vd, q_start, none, table, mask).shape == (0, 4, 64)
    assert bool((g.kv_weigh(ctx, q, kd, q_start, none, table, lse, w) == 1).all())
    index, counts = g.kv_select(ctx, w, none, table, 4)
    assert index.shape == (0, 2, 4) and counts.shape == (0,)
    assert g.kv_compact(ctx, kd, vd, none, table, index, counts).shape == (0,)
    one, page = torch.tensor([20], dtype=torch.int32, device="cuda"), torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    index, counts = g.kv_select(ctx, w, one, page, 0)
    assert counts.tolist() == [0]
    assert g.kv_compact(ctx, kd, vd, one, page, index, counts).tolist() == [0]
    a, codes, scales, zeros, _ = (x.cuda() if x is not None else None for x in w4_inputs(3, 16, 64, 64, F16, True))
    assert g.w4_gemm(ctx, a[:0], codes, scales, zeros).shape == (0, 16)
    assert g.w4_gemm(ctx, a, codes[:0], scales[:0], zeros[:0]).shape == (3, 0)
    clean(ctx)
    assert torch.equal(kd, vd)
