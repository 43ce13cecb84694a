"""Attention over the paged cache against 64 bits: ragged batches, masks, pages, shared prefixes,
layouts, stale rows, captured graphs, streams, refusals, and a whole serving step."""
import ctypes
import math

import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from serving_ref import TYPES, attention, batch, check_attention, check_rope, rope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ctx():
    from tensor_core_gemm_tcgen05_gb300 import _build
    _build.build()
    c = g.Context(0)
    yield c
    c.close()


def normal(shape, seed, t):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(t)


def dev(x):
    return None if x is None else x.to(DEV)


def done(ctx):
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_OK, 0)


def problem(n_q, kv, dtype="float16", hq=8, hk=2, d=128, page=16, prefix=0, by_rows=False, spare=0, seed=0, stale=math.nan):
    """Queries and a cache whose rows past every sequence's end (and unused pages) hold `stale`."""
    t = TYPES[dtype]
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=seed)
    q = normal((sum(n_q) + spare, hq, d), seed + 1, t)
    k, v = (normal((b["pages"], hk, page, d), seed + 2 + i, t) for i in range(2))
    if stale is not None:
        used = torch.zeros(b["pages"], page, dtype=torch.bool)
        if prefix:
            used[b["prefix_pages"].long()] = True
        for s, n in enumerate(kv):
            for i in range(0, n, page):
                used[int(b["page_table"][s, i // page]), : min(page, n - i)] = True
        for x in (k, v):
            x.transpose(1, 2)[~used] = stale
    kd, vd = dev(k), dev(v)
    if by_rows:
        kd, vd = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kd, vd))
    return b, q, k, v, kd, vd


def run(ctx, b, q, kd, vd, max_q=None, scale=None):
    tokens, hq, d = q.shape
    # outputs filled with a mark, with guard rows behind them
    guard = torch.full((tokens + 2, hq, d), 7.0, dtype=q.dtype, device=DEV)
    guard_lse = torch.full((tokens + 2, hq), 7.0, dtype=torch.float32, device=DEV)
    out, lse = guard[:tokens], guard_lse[:tokens]
    g.paged_attention(ctx, dev(q), kd, vd, dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]), max_q=max_q,
                      prefix_pages=dev(b["prefix_pages"]), scale=scale, out=out, lse=lse)
    done(ctx)
    assert torch.all(guard[tokens:] == 7.0) and torch.all(guard_lse[tokens:] == 7.0)
    n = int(b["q_start"][-1])
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0), "wrote tokens of no sequence"
    return out[:n].cpu(), lse[:n].cpu()


def check(ctx, p, what, max_q=None, scale=None):
    b, q, k, v, kd, vd = p
    n = int(b["q_start"][-1])
    s = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    ref, lse, spread = attention(q[:n], torch.nan_to_num(k.float(), 0, 0, 0), torch.nan_to_num(v.float(), 0, 0, 0), b, s, DEV)
    got, got_lse = run(ctx, b, q, kd, vd, max_q=max_q, scale=scale)
    check_attention(got, got_lse, ref, lse, spread, what)
    return got


# lengths: one token and long ones, odd sizes, empty sequences, more new tokens than keys (rows
# that see nothing), ends inside pages and blocks
LENS = {
    "one_key": ([1], [1]),
    "one_token": ([1], [777]),
    "no_keys": ([1, 2], [0, 0]),
    "decode": ([1] * 9, [1, 63, 64, 65, 128, 129, 500, 17, 1000]),
    "drafts": ([3, 0, 1, 2, 4], [3, 100, 64, 200, 67]),
    "rows_without_keys": ([5, 40, 1], [2, 20, 0]),
    "prompt": ([300], [300]),
    "prompt_odd": ([257, 1, 129], [257, 1, 129]),
    "pieces": ([200, 1, 70], [900, 333, 70]),
    "edges": ([128, 256, 64, 16, 17], [128, 512, 65, 16, 31]),
}


@pytest.mark.parametrize("dtype,hq,hk,d,page,by_rows", [
    ("float16", 8, 2, 128, 16, False), ("bfloat16", 8, 8, 128, 64, True), ("float16", 4, 1, 64, 32, True),
    ("bfloat16", 14, 2, 64, 256, False), ("float16", 3, 1, 128, 128, False), ("bfloat16", 40, 5, 128, 1024, False)], ids=str)
@pytest.mark.parametrize("lens", list(LENS))
def test_matches_64_bits(ctx, lens, dtype, hq, hk, d, page, by_rows):
    n_q, kv = LENS[lens]
    p = problem(n_q, kv, dtype, hq, hk, d, page, by_rows=by_rows, spare=3, seed=len(lens))
    check(ctx, p, lens)
    check(ctx, p, lens + ", max_q given", max_q=max(n_q))


@pytest.mark.parametrize("group", [1, 2, 5, 7, 16, 32, 64, 100, 128])
def test_heads_per_key_head(ctx, group):
    check(ctx, problem([3, 1, 20], [100, 1, 200], hq=2 * group, hk=2), group)


@pytest.mark.parametrize("max_q", [0, 1, 2, 1000])
def test_results_do_not_depend_on_max_q(ctx, max_q):
    check(ctx, problem([150, 1, 3], [200, 300, 3], hq=4, hk=1), max_q, max_q=max_q)


@pytest.mark.parametrize("n_q,kv,hq,hk,d,page,prefix", [
    ([1] * 20, [1 + 13 * i for i in range(20)], 8, 2, 128, 16, 9),      # one tile of rows for the prefix
    ([1] * 100, [1 + i % 7 for i in range(100)], 8, 1, 128, 32, 40),    # several tiles
    ([2, 1, 0, 3, 1], [2, 50, 10, 3, 1], 4, 2, 64, 64, 3),
    ([1] * 4, [0, 1, 0, 5], 8, 2, 128, 16, 5),                          # tokens that stand inside the prefix
    ([40, 1, 3], [10, 1, 2], 4, 1, 64, 16, 2),                          # ... and some before it
    ([300, 2], [300, 2], 8, 2, 128, 64, 3),                             # not joint: the prefix is read with the own keys
    ([1], [5], 8, 2, 128, 16, 30),
    ([0, 0, 1], [0, 3, 4], 2, 2, 64, 128, 1),
    ([1] * 130, [200] * 130, 5, 1, 128, 32, 12),                        # more tiles than share a launch
    ([2] * 30 + [90, 1], [500] * 30 + [90, 7], 4, 2, 64, 16, 33)], ids=lambda v: str(v)[:40])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_shared_prefix(ctx, n_q, kv, hq, hk, d, page, prefix, dtype):
    p = problem(n_q, kv, dtype, hq, hk, d, page, prefix=prefix, spare=1, seed=7)
    check(ctx, p, (n_q, prefix), max_q=max(n_q))   # (what is known decides whether one launch takes all keys)
    check(ctx, p, (n_q, prefix))


def test_many_sequences(ctx):
    """More sequences than threads per CTA, and empty ones among them."""
    n = 1500
    n_q = [1 if i % 5 else 0 for i in range(n)]
    kv = [a + (i * 7) % 90 for i, a in enumerate(n_q)]
    check(ctx, problem(n_q, kv, hq=2, hk=1, d=64), "many")


@pytest.mark.parametrize("lens", [([1], [40000]), ([1, 1, 1], [9000, 1, 20000]), ([5], [30000]), ([2000, 1], [2600, 5000])], ids=str)
def test_long_keys_are_split_and_joined(ctx, lens):
    check(ctx, problem(*lens, hq=8, hk=2, page=64), lens)


def test_large_scores_and_rising_maximum(ctx):
    """Scores that grow along the keys by far more than the threshold at which rows are rescaled."""
    b, q, k, v, kd, vd = problem([3, 140], [700, 700], hq=4, hk=2, stale=None)
    ramp = torch.linspace(0, 6, 700)
    for s in range(2):
        for i in range(700):
            k[int(b["page_table"][s, i // 16]), :, i % 16] *= float(ramp[i])
    check(ctx, (b, q, k, v, dev(k), dev(v)), "ramp")
    check(ctx, (b, q, k, v, dev(k), dev(v)), "negative scale", scale=-0.3)


def test_zero_scale_is_the_mean(ctx):
    check(ctx, problem([1, 5], [100, 64]), "scale 0", scale=0.0)


@pytest.mark.parametrize("stale", [math.nan, math.inf, -math.inf, 65504.0])
def test_stale_rows_leave_no_trace(ctx, stale):
    a = problem([1, 3, 150], [70, 35, 170], page=64, stale=stale)
    check(ctx, a, stale)


def test_strided_queries_and_outputs(ctx):
    """Queries in a packed projection, head-major outputs, a padded lse."""
    b, q, k, v, kd, vd = problem([2, 30, 1], [50, 30, 129], hq=6, hk=3)
    n, hq, d = q.shape
    packed = torch.zeros(n, (hq + 6) * d, dtype=q.dtype, device=DEV)
    view = packed[:, 2 * d : (hq + 2) * d].unflatten(1, (hq, d))
    view.copy_(q)
    out = torch.full((hq, n + 1, d), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((n, hq + 5), 7.0, device=DEV)
    g.paged_attention(ctx, view, kd, vd, dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]),
                      out=out[:, :n].transpose(0, 1), lse=lse[:, :hq])
    done(ctx)
    ref, rl, spread = attention(q, torch.nan_to_num(k.float()), torch.nan_to_num(v.float()), b, d ** -0.5)
    check_attention(out[:, :n].transpose(0, 1).cpu(), lse[:, :hq].cpu(), ref, rl, spread, "strided")
    assert torch.all(out[:, n] == 7.0) and torch.all(lse[:, hq:] == 7.0)


def test_pages_may_be_shared_between_sequences(ctx):
    b, q, k, v, kd, vd = problem([1, 1, 1], [60, 60, 60], stale=None)
    b["page_table"][1, :3] = b["page_table"][0, :3]
    b["page_table"][2] = b["page_table"][0]
    check(ctx, (b, q, k, v, kd, vd), "shared pages")


def test_one_tensor_of_keys_and_values_and_a_wide_table(ctx):
    b, q, k, v, kd, vd = problem([1, 2], [40, 50], hk=2, page=32)
    both = torch.stack((kd, vd), 1)
    wide = torch.full((2, 50), 2 ** 31 - 1, dtype=torch.int32)
    wide[:, : b["page_table"].shape[1]] = b["page_table"]
    b["page_table"] = wide
    check(ctx, (b, q, k, v, both[:, 0], both[:, 1]), "one tensor")


def test_same_bits_again(ctx):
    b, q, k, v, kd, vd = problem([1, 4, 200], [3000, 2500, 900], prefix=20)
    one = run(ctx, b, q, kd, vd)
    for _ in range(3):
        two = run(ctx, b, q, kd, vd)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_captured_graph_follows_new_lengths(ctx):
    """Two graphs with workspaces of their own, replayed on two streams at once with lengths that
    change between replays."""
    graphs = []
    for i in range(2):
        b, q, k, v, kd, vd = problem([1, 1, 1], [300, 300, 300], seed=10 * i, stale=None)
        qd, qs, kv, pt = dev(q), dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"])
        out, lse = torch.empty_like(qd), torch.empty(3, 8, device=DEV)
        need = g.paged_attention_workspace(ctx, qd, kd, vd, qs, kv, pt, max_q=1)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        args = (ctx, qd, kd, vd, qs, kv, pt)
        with torch.cuda.stream(stream):
            g.paged_attention(*args, max_q=1, out=out, lse=lse, workspace=ws)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                g.paged_attention(*args, max_q=1, out=out, lse=lse, workspace=ws)
        graphs.append((b, q, k, v, kv, out, lse, stream, graph, ws))
    torch.cuda.synchronize()
    for lens in ([1, 2, 3], [300, 1, 64], [0, 128, 299]):
        for b, q, k, v, kv, out, lse, stream, graph, _ in graphs:
            kv.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for x in graphs:
                with torch.cuda.stream(x[7]):
                    x[8].replay()
        done(ctx)
        for b, q, k, v, kv, out, lse, *_ in graphs:
            ref, rl, spread = attention(q, k, v, {**b, "kv": lens}, 128 ** -0.5)
            check_attention(out.cpu(), lse.cpu(), ref, rl, spread, lens)


def test_another_stream_allocates_its_own_workspace(ctx):
    b, q, k, v, kd, vd = problem([1, 1], [5000, 300])
    ref, rl, spread = attention(q, torch.nan_to_num(k.float()), torch.nan_to_num(v.float()), b, 128 ** -0.5)
    qd, args = dev(q), (dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for i in range(6):   # calls on two streams at once
        lse = torch.empty(2, 8, device=DEV)
        outs.append((g.paged_attention(ctx, qd, kd, vd, *args, lse=lse, stream=side if i % 2 else None), lse))
    done(ctx)
    for out, lse in outs:
        check_attention(out.cpu(), lse.cpu(), ref, rl, spread, "streams")


@pytest.mark.parametrize("what", ["page", "page_negative", "kv_long", "kv_negative", "q_start", "prefix_page"])
def test_bad_batches_are_reported_and_do_no_harm(ctx, what):
    """Indexes out of range are limited by the kernel's own checks; other sequences are right."""
    b, q, k, v, kd, vd = problem([1, 1, 1], [100, 200, 50], prefix=2 if what == "prefix_page" else 0, stale=None)
    bad = {x: y.clone() if torch.is_tensor(y) else y for x, y in b.items()}
    if what == "page":
        bad["page_table"][1, 1] = b["pages"]
    elif what == "page_negative":
        bad["page_table"][1, 1] = -2 ** 31
    elif what == "kv_long":
        bad["kv_lens"][1] = 2 ** 31 - 1
        bad["page_table"][1] = 0
    elif what == "kv_negative":
        bad["kv_lens"][1] = -7
    elif what == "q_start":
        bad["q_start"][3] = 1000
    else:
        bad["prefix_pages"][1] = 2 ** 30
    out = g.paged_attention(ctx, dev(q), kd, vd, dev(bad["q_start"]), dev(bad["kv_lens"]), dev(bad["page_table"]),
                            prefix_pages=dev(bad["prefix_pages"]))
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_ERR_INDEX, 8)
    if what != "prefix_page":
        ref, _, spread = attention(q, k, v, b, 128 ** -0.5)
        for i in (0, 2):
            assert torch.all((out[i].cpu().double() - ref[i]).abs() <= 2.0 ** -10 * ref[i].abs() + 2.0 ** -10 * spread[i])
    # and the context is as good as before
    check(ctx, problem([2], [70]), "after")


def test_refusals(ctx):
    from tensor_core_gemm_tcgen05_gb300.serving import Heads, KvBatch, KvCache, Rope
    L, h = g.lib(), ctx.handle
    t, T, hq, hk, d, page, pages = torch.float16, 3, 4, 2, 128, 16, 6
    q, out = (torch.zeros(T, hq, d, dtype=t, device=DEV) for _ in range(2))
    k, v = (torch.zeros(T, hk, d, dtype=t, device=DEV) for _ in range(2))
    kc, vc = (torch.zeros(pages, hk, page, d, dtype=t, device=DEV) for _ in range(2))
    qs, kv = torch.tensor([0, 3], dtype=torch.int32, device=DEV), torch.tensor([3], dtype=torch.int32, device=DEV)
    pt = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    table = g.rope_table(d)[0].to(DEV)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    host = torch.zeros(4096, dtype=t)
    hp = (host.data_ptr() + 15) // 16 * 16
    stream = torch.cuda.current_stream().cuda_stream

    def heads(x, **kw):
        return Heads(**{**dict(data=x.data_ptr(), heads=x.shape[1], token_stride=x.stride(0), head_stride=x.stride(1)), **kw})

    def cache(**kw):
        return KvCache(**{**dict(k=kc.data_ptr(), v=vc.data_ptr(), num_pages=pages, page_size=page, kv_heads=hk, head_dim=d,
                                 page_stride=kc.stride(0), head_stride=kc.stride(1), row_stride=kc.stride(2), dtype=0), **kw})

    def bt(**kw):
        return KvBatch(**{**dict(num_seqs=1, num_tokens=T, max_q=0, q_start=qs.data_ptr(), kv_lens=kv.data_ptr(),
                                 page_table=pt.data_ptr(), table_width=4, table_stride=4, prefix_pages=None, num_prefix_pages=0), **kw})

    def rp(**kw):
        return Rope(**{**dict(table=table.data_ptr(), rotary_dim=d, q_norm=None, k_norm=None, eps=1e-6, scale=1.0, interleaved=0), **kw})

    def at(x):
        return ctypes.byref(x)

    def attend(c=None, b=None, hq_=None, ho=None, scale=0.1, lse=None, stride=0, w=ws.data_ptr(), n=ws.numel()):
        return L.gemm_paged_attention(h, at(c or cache()), at(b or bt()), at(hq_ or heads(q)), scale, at(ho or heads(out)), lse,
                                      stride, w, n, stream)

    def append(c=None, b=None, **kw):
        a = {**dict(q=heads(q), k=heads(k), v=heads(v), r=rp(), o=heads(out)), **kw}
        return L.gemm_kv_append(h, at(c or cache()), at(b or bt()), at(a["q"]), at(a["k"]), at(a["v"]), at(a["r"]), at(a["o"]), stream)

    def rope_(**kw):
        a = {**dict(dtype=0, T=T, d=d, q=heads(q), k=heads(k), p=pos.data_ptr(), r=rp(), qo=heads(out), ko=heads(v)), **kw}
        return L.gemm_qk_rope(h, a["dtype"], a["T"], a["d"], at(a["q"]), at(a["k"]), a["p"], at(a["r"]), at(a["qo"]), at(a["ko"]), stream)

    ARG, ALIGN, DEVICE, OK = g.GEMM_ERR_ARG, g.GEMM_ERR_ALIGN, g.GEMM_ERR_DEVICE, g.GEMM_OK
    assert attend() == OK and append() == OK and rope_() == OK
    # the cache
    for kw in (dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(page_size=0), dict(head_dim=96), dict(head_dim=256),
               dict(dtype=2), dict(num_pages=0), dict(num_pages=2 ** 31), dict(kv_heads=0), dict(k=None), dict(row_stride=0),
               dict(head_stride=-8), dict(page_stride=2 ** 41), dict(v=kc.data_ptr()), dict(row_stride=64), dict(page_stride=8)):
        assert attend(c=cache(**kw)) == ARG, kw
        assert append(c=cache(**kw)) == ARG, kw
    for kw in (dict(k=kc.data_ptr() + 2), dict(row_stride=d + 4)):
        assert attend(c=cache(**kw)) == ALIGN and append(c=cache(**kw)) == ALIGN, kw
    assert attend(c=cache(k=hp)) == DEVICE and append(c=cache(v=hp)) == DEVICE
    # the batch
    for kw in (dict(num_seqs=-1), dict(num_tokens=-1), dict(num_tokens=2 ** 31), dict(q_start=None), dict(kv_lens=None), dict(page_table=None),
               dict(table_width=2 ** 28), dict(table_width=-1), dict(table_stride=-4), dict(max_q=-1), dict(num_prefix_pages=-1),
               dict(num_prefix_pages=2 ** 27)):
        assert attend(b=bt(**kw)) == ARG, kw
        assert append(b=bt(**kw)) == ARG, kw
    assert attend(b=bt(num_prefix_pages=2)) == ARG   # no pages given
    assert attend(b=bt(q_start=qs.data_ptr() + 1)) == ALIGN and append(b=bt(kv_lens=kv.data_ptr() + 2)) == ALIGN
    assert attend(b=bt(page_table=hp)) == DEVICE and append(b=bt(q_start=hp)) == DEVICE
    # heads
    assert attend(hq_=heads(q, heads=3), ho=heads(out, heads=3)) == ARG      # not a multiple of the key heads
    assert attend(hq_=heads(q, heads=2)) == ARG                              # not the outputs'
    assert attend(ho=heads(q)) == ARG                                        # out over q
    assert attend(ho=heads(out, data=kc.data_ptr())) == ARG
    assert attend(hq_=heads(q, token_stride=0)) == ARG                       # broadcast
    assert attend(hq_=heads(q, head_stride=d + 4)) == ALIGN
    assert attend(hq_=heads(q, data=q.data_ptr() + 8)) == ALIGN
    assert attend(hq_=heads(q, data=hp)) == DEVICE
    assert append(k=heads(k, heads=1)) == ARG and append(o=heads(out, heads=2)) == ARG
    assert append(k=heads(k, data=kc.data_ptr())) == ARG and append(o=heads(v, heads=4)) == ARG
    assert append(q=heads(q, heads=0), o=heads(out, heads=0)) == OK
    # the rest
    assert attend(scale=math.nan) == ARG and attend(scale=math.inf) == ARG
    assert attend(w=None) == ARG and attend(n=100) == ARG and attend(w=ws.data_ptr() + 16) == ALIGN
    assert attend(lse=ws.data_ptr() + 64, stride=hq) == ARG                  # inside the workspace
    assert attend(lse=ws.data_ptr() + ws.numel() - 4096, stride=1) == ARG    # rows over each other
    for kw in (dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16), dict(table=None), dict(scale=math.inf), dict(eps=-1.0),
               dict(interleaved=2)):
        assert rope_(r=rp(**kw)) == ARG and append(r=rp(**kw)) == ARG, kw
    assert rope_(r=rp(table=table.data_ptr() + 4)) == ALIGN and rope_(r=rp(q_norm=q.data_ptr() + 2)) == ALIGN
    assert rope_(r=rp(table=hp)) == DEVICE
    assert rope_(dtype=5) == ARG and rope_(d=80) == ARG and rope_(T=-1) == ARG and rope_(p=None) == ARG and rope_(p=hp) == DEVICE
    assert rope_(qo=heads(q, data=q.data_ptr() + 2 * d)) == ARG and rope_(ko=heads(q, heads=2)) == ARG
    assert rope_(T=0, p=None) == OK and rope_(qo=heads(q)) == OK
    # nothing to do
    assert attend(b=bt(num_tokens=0)) == OK and append(b=bt(num_seqs=0)) == OK
    assert L.gemm_paged_attention_workspace(h, at(cache()), at(bt(num_tokens=0)), 4) == 0
    assert L.gemm_paged_attention_workspace(h, at(cache()), at(bt()), 5) == ARG
    assert 0 < L.gemm_paged_attention_workspace(h, at(cache()), at(bt(q_start=None)), 4) <= ws.numel()
    done(ctx)


@pytest.mark.parametrize("n_q,kv", [([1, 1], [300, 2000]), ([300], [500])], ids=str)
def test_timeout_then_recovery(ctx, n_q, kv):
    """A held back first load: the wait for it runs out, the kernel ends, the call after it is right."""
    b, q, k, v, kd, vd = problem(n_q, kv)
    args = (dev(q), kd, vd, dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]))
    g.gemm_set_timeout_ns(ctx, 20 * 10 ** 6)
    g.gemm_set_debug(ctx, g.GEMM_DEBUG_WITHHOLD_FIRST_LOAD)
    try:
        g.paged_attention(ctx, *args)
        torch.cuda.synchronize()
        status, detail = g.gemm_last_device_error(ctx)
        assert status == g.GEMM_ERR_TIMEOUT and detail in (1, 2, 3, 4)
    finally:
        g.gemm_set_debug(ctx, g.GEMM_DEBUG_NONE)
        g.gemm_set_timeout_ns(ctx, 2 * 10 ** 9)
    check(ctx, (b, q, k, v, kd, vd), "after a timeout")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_serving_steps(ctx, dtype):
    """Prompts, then decoding steps, as a serving loop runs them: projection (GEMM), append with
    norm and rotation, attention over the cache behind a shared prefix."""
    t = TYPES[dtype]
    hq, hk, d, page, width, prefix = 8, 2, 128, 16, 256, 2
    prompts, steps = [5, 30, 1], 3
    total = [n + steps for n in prompts]
    b0 = batch(prompts, total, page, prefix_pages=prefix, seed=3)
    kc, vc = (torch.full((b0["pages"], hk, page, d), math.nan, dtype=t) for _ in range(2))
    pre = [normal((prefix, hk, page, d), 40 + i, t) for i in range(2)]
    kc[b0["prefix_pages"].long()], vc[b0["prefix_pages"].long()] = pre
    kd, vd = dev(kc), dev(vc)
    table, _ = g.rope_table(d, 500000.0)
    wq, wk = normal((d,), 50, t), normal((d,), 51, t)
    weight = (normal((width, (hq + 2 * hk) * d), 52, torch.float32) / width ** 0.5).half()
    lens = list(prompts)
    n_q = list(prompts)
    for step in range(steps + 1):
        b = dict(b0, n_q=n_q, kv=list(lens), q_start=torch.tensor([sum(n_q[:i]) for i in range(4)], dtype=torch.int32),
                 kv_lens=torch.tensor(lens, dtype=torch.int32))
        x = normal((sum(n_q), width), 60 + step, torch.float16)
        qkv = g.gemm(ctx, dev(x), dev(weight)).to(t)   # the library's projection, FP16
        q, k, v = (y.unflatten(1, (-1, d)) for y in qkv.split([hq * d, hk * d, hk * d], 1))
        args = (dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]))
        qr = g.kv_append(ctx, q, k, v, kd, vd, *args, dev(table), prefix_len=prefix * page, q_norm=dev(wq), k_norm=dev(wk))
        lse = torch.empty(sum(n_q), hq, device=DEV)
        out = g.paged_attention(ctx, qr, kd, vd, *args, max_q=max(n_q), prefix_pages=dev(b["prefix_pages"]), lse=lse)
        done(ctx)
        # the same from the tensors in between (each stage's rounded outputs feed the next)
        pos = [prefix * page + lens[s] - n_q[s] + i for s in range(3) for i in range(n_q[s])]
        check_rope(qr.cpu(), *rope(q.cpu(), wq, pos, table, False, 1.0, 1e-6), "queries")
        ref, rl, spread = attention(qr.cpu(), torch.nan_to_num(kd.cpu()), torch.nan_to_num(vd.cpu()), b, d ** -0.5)
        check_attention(out.cpu(), lse.cpu(), ref, rl, spread, step)
        n_q = [1, 1, 1]
        lens = [x + 1 for x in lens]
