"""The serving operators at the ends of what their documentation allows: batches that begin behind
the first token, batches without keys or tokens, offsets past 32 bits, sizes at their limits,
threads that call at once, one captured step of both operators."""
import math
import threading

import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from tensor_core_gemm_tcgen05_gb300 import serving
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


def normal(shape, seed, t=torch.float16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(t)


def done(ctx):
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_OK, 0)


def on_device(b):
    return b["q_start"].to(DEV), b["kv_lens"].to(DEV), b["page_table"].to(DEV)


@pytest.mark.parametrize("n_q,kv,prefix,max_q", [([1, 1, 1], [70, 300, 5], 0, 1), ([200, 3], [230, 90], 0, None),
                                                 ([1] * 6, [9, 0, 40, 1, 64, 65], 3, 1), ([150, 2, 90], [150, 5, 200], 2, None),
                                                 ([300] * 3, [300] * 3, 40, 300)], ids=str)
def test_tokens_before_the_first_sequence_are_left_alone(ctx, n_q, kv, prefix, max_q):
    lead, behind, hq, hk, d, page = 37, 3, 8, 2, 128, 16
    n_kv = [max(a, b) for a, b in zip(n_q, kv)]
    b = batch(n_q, n_kv, page, prefix_pages=prefix, seed=4)
    tokens = sum(n_q)
    q = normal((lead + tokens + behind, hq, d), 1)
    kn, vn = normal((lead + tokens + behind, hk, d), 2), normal((lead + tokens + behind, hk, d), 3)
    k, v = normal((b["pages"], hk, page, d), 4), normal((b["pages"], hk, page, d), 5)
    kd, vd = k.to(DEV), v.to(DEV)
    starts = (b["q_start"] + lead).to(DEV)
    lens, table = b["kv_lens"].to(DEV), b["page_table"].to(DEV)
    q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    g.kv_append(ctx, q.to(DEV), kn.to(DEV), vn.to(DEV), kd, vd, starts, lens, table, g.rope_table(d)[0].to(DEV),
                prefix_len=prefix * page, q_out=q_out)
    out, lse = torch.full_like(q_out, 7.0), torch.full((q.shape[0], hq), 7.0, device=DEV)
    pages = b["prefix_pages"].to(DEV) if prefix else None
    g.paged_attention(ctx, q_out, kd, vd, starts, lens, table, max_q=max_q, prefix_pages=pages, out=out, lse=lse)
    done(ctx)
    for x in (q_out, out, lse):
        assert torch.all(x[:lead] == 7.0) and torch.all(x[lead + tokens :] == 7.0)
    mine = slice(lead, lead + tokens)
    pos = [prefix * page + n_kv[s] - n_q[s] + i for s in range(len(n_q)) for i in range(n_q[s])]
    check_rope(q_out[mine].cpu(), *rope(q[mine], None, pos, g.rope_table(d)[0], False, 1.0, 1e-6), "queries")
    ref, rl, spread = attention(q_out[mine].cpu(), kd.cpu(), vd.cpu(), b, d ** -0.5)
    check_attention(out[mine].cpu(), lse[mine].cpu(), ref, rl, spread, "attention")


@pytest.mark.parametrize("max_q", [None, 1, 300])
@pytest.mark.parametrize("width", [0, 2])
def test_no_keys_at_all(ctx, width, max_q):
    """New tokens in front of every key: nothing is seen, no page is read."""
    n_q = [1, 300, 0, 2]
    q = normal((303, 4, 64), 1).to(DEV)
    cache = torch.full((3, 2, 16, 64), math.nan, dtype=torch.float16, device=DEV)
    starts = torch.tensor([0, 1, 301, 301, 303], dtype=torch.int32, device=DEV)
    lens = torch.zeros(4, dtype=torch.int32, device=DEV)
    table = torch.full((4, width), -5, dtype=torch.int32, device=DEV)
    lse = torch.zeros(303, 4, device=DEV)
    out = g.paged_attention(ctx, q, cache, cache.clone(), starts, lens, table, max_q=max_q, lse=lse)
    done(ctx)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


def test_nothing_to_do(ctx):
    cache = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    other = torch.zeros_like(cache)
    q, k = (torch.empty(0, h, 128, dtype=torch.bfloat16, device=DEV) for h in (4, 2))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    for starts, lens, t in ((ints(0, 0, 0, 0), ints(5, 0, 16), table), (ints(0), ints(), table[:0])):
        assert g.kv_append(ctx, q, k, k, cache, other, starts, lens, t).shape == q.shape
        assert g.paged_attention(ctx, q, cache, other, starts, lens, t, lse=torch.empty(0, 4, device=DEV)).shape == q.shape
        assert g.paged_attention_workspace(ctx, q, cache, other, starts, lens, t) == 0
    assert g.qk_rope(ctx, q, k, ints())[1].shape == k.shape
    done(ctx)


@pytest.mark.parametrize("prefix", [0, 2])
def test_offsets_past_32_bits(ctx, prefix):
    """Pages 2^30 elements apart, heads 2^28, keys and values in one allocation of about 20 GB."""
    n_q, kv, hq, hk, d, page = [1, 40, 3], [30, 75, 3], 8, 2, 64, 16
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=6, spare=0)
    space = torch.empty(b["pages"] * 2 ** 30 + 2 ** 16, dtype=torch.bfloat16, device=DEV)
    kd, vd = (space.as_strided((b["pages"], hk, page, d), (2 ** 30, 2 ** 28, 2 ** 10, 1), at) for at in (0, 2 ** 29))
    tokens = sum(n_q)
    q, k, v = (normal((tokens, h, d), i, torch.bfloat16) for i, h in enumerate((hq, hk, hk)))
    first, second = (normal(kd.shape, 7 + i, torch.bfloat16) for i in range(2))
    kd.copy_(first)
    vd.copy_(second)
    args = on_device(b)
    q_out = g.kv_append(ctx, q.to(DEV), k.to(DEV), v.to(DEV), kd, vd, *args, g.rope_table(d)[0].to(DEV), prefix_len=prefix * page)
    lse = torch.empty(tokens, hq, device=DEV)
    out = g.paged_attention(ctx, q_out, kd, vd, *args, prefix_pages=b["prefix_pages"].to(DEV) if prefix else None, lse=lse)
    done(ctx)
    for s in range(3):
        for i in range(n_q[s]):
            place = kv[s] - n_q[s] + i
            row = vd[int(b["page_table"][s, place // page]), :, place % page].cpu()
            assert torch.equal(row, v[int(b["q_start"][s]) + i])
    ref, rl, spread = attention(q_out.cpu(), kd.cpu(), vd.cpu(), b, d ** -0.5)
    check_attention(out.cpu(), lse.cpu(), ref, rl, spread, "far")


def test_sizes_at_their_limits(ctx):
    """A table of as many keys as a call takes (of which a sequence has few), and one page more."""
    page, hk, d = 1024, 1, 64
    width = 2 ** 31 // page - 1
    b = batch([1], [1500], page, seed=2)
    k, v = normal((b["pages"], hk, page, d), 1), normal((b["pages"], hk, page, d), 2)
    q = normal((1, 2, d), 3)
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    table[:, :2] = b["page_table"].to(DEV)
    lse = torch.empty(1, 2, device=DEV)
    args = (q.to(DEV), k.to(DEV), v.to(DEV), b["q_start"].to(DEV), b["kv_lens"].to(DEV))
    out = g.paged_attention(ctx, *args, table, lse=lse)
    done(ctx)
    ref, rl, spread = attention(q, k, v, b, d ** -0.5)
    check_attention(out.cpu(), lse.cpu(), ref, rl, spread, "limit")
    more = torch.full((1, width + 1), -1, dtype=torch.int32, device=DEV)
    with pytest.raises(g.GemmError) as e:
        g.paged_attention(ctx, *args, more)
    assert e.value.status == g.GEMM_ERR_ARG
    done(ctx)


def test_threads_that_call_at_once(ctx):
    """Two threads, a stream each, one context; each call its own workspace."""
    shapes = [([1] * 20, [100 + 37 * i for i in range(20)]), ([130, 1, 64], [400, 2000, 64])]
    jobs = []
    for i, (n_q, kv) in enumerate(shapes):
        b = batch(n_q, kv, 32, seed=i)
        q, k, v = normal((sum(n_q), 8, 128), 1), normal((b["pages"], 2, 32, 128), 2), normal((b["pages"], 2, 32, 128), 3)
        ref = attention(q, k, v, b, 128 ** -0.5)
        jobs.append((b, [x.to(DEV) for x in (q, k, v)], on_device(b), ref, []))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        try:
            b, (q, k, v), args, _, outs = job
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    lse = torch.empty(q.shape[0], 8, device=DEV)
                    outs.append((g.paged_attention(ctx, q, k, v, *args, max_q=max(b["n_q"]), lse=lse), lse))
            stream.synchronize()
        except Exception as e:   # told in the main thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    done(ctx)
    assert not failed
    for _, _, _, ref, outs in jobs:
        for out, lse in outs:
            check_attention(out.cpu(), lse.cpu(), *ref, "threads")


def test_captured_step_of_both_operators(ctx):
    """Append and attention in one graph, the lengths advanced on the device between replays."""
    steps, hq, hk, d, page = 4, 4, 2, 64, 16
    kv = [13, 15, 47]
    b = batch([1, 1, 1], [n + steps for n in kv], page, seed=9)
    k, v = normal((b["pages"], hk, page, d), 1), normal((b["pages"], hk, page, d), 2)
    kd, vd = k.to(DEV), v.to(DEV)
    starts, _, table = on_device(b)
    lens = torch.tensor(kv, dtype=torch.int32, device=DEV)
    words = g.rope_table(d, 10000.0)[0].to(DEV)
    q, kn, vn = (normal((3, h, d), 3 + i).to(DEV) for i, h in enumerate((hq, hk, hk)))
    q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(3, hq, device=DEV)
    ws = torch.empty(g.paged_attention_workspace(ctx, q, kd, vd, starts, lens, table, max_q=1), dtype=torch.uint8, device=DEV)

    def step():
        lens.add_(1)
        g.kv_append(ctx, q, kn, vn, kd, vd, starts, lens, table, words, q_out=q_out)
        g.paged_attention(ctx, q_out, kd, vd, starts, lens, table, max_q=1, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step()
    for i in range(1, steps + 1):
        new = [normal((3, h, d), 10 * i + j) for j, h in enumerate((hq, hk, hk))]
        for x, y in zip((q, kn, vn), new):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        done(ctx)
        now = [n + i for n in kv]
        for s in range(3):
            row = vd[int(b["page_table"][s, (now[s] - 1) // page]), :, (now[s] - 1) % page].cpu()
            assert torch.equal(row, new[2][s])
        check_rope(q_out.cpu(), *rope(new[0], None, [n - 1 for n in now], words.cpu(), False, 1.0, 1e-6), i)
        ref, rl, spread = attention(q_out.cpu(), kd.cpu(), vd.cpu(), {**b, "kv": now}, d ** -0.5)
        check_attention(out.cpu(), lse.cpu(), ref, rl, spread, i)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan], ids=str)
@pytest.mark.parametrize("n_q,kv,hq,hk,d,page,prefix,max_q", [
    ([3, 1, 2], [70, 1, 64], 8, 2, 64, 16, 0, 3), ([300], [300], 8, 2, 128, 16, 0, None), ([5, 40, 1], [2, 20, 9], 8, 8, 128, 32, 0, 40),
    ([200, 3, 64], [1000, 67, 64], 6, 2, 64, 64, 0, None), ([4] * 9, [30] * 9, 4, 1, 128, 16, 5, 4), ([150], [150], 2, 2, 64, 16, 3, None),
    ([20] * 6, [3, 9, 20, 21, 1, 50], 4, 2, 128, 16, 4, 20), ([300] * 3, [100, 300, 250], 8, 2, 64, 16, 20, 300)], ids=str)
def test_values_that_are_not_finite_reach_those_that_see_them_only(ctx, n_q, kv, hq, hk, d, page, prefix, max_q, bad):
    """In a sequence's new keys, which its earlier new tokens do not see (and in an old one, which all
    do), and in the last keys of a prefix, which tokens inside it do not see."""
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=8)
    tokens = sum(n_q)
    q = normal((tokens, hq, d), 1)
    k, v = normal((b["pages"], hk, page, d), 2), normal((b["pages"], hk, page, d), 3)
    gen = torch.Generator().manual_seed(5)
    marks = []   # (sequence, own key, head, dim)
    for s, n in enumerate(kv):
        for _ in range(min(n, 3)):
            j = n - 1 - int(torch.randint(0, min(n, n_q[s] + 1), (1,), generator=gen))
            marks.append((s, j, int(torch.randint(0, hk, (1,), generator=gen)), int(torch.randint(0, d, (1,), generator=gen))))
    zeroed = v.clone()
    for s, j, h, e in marks:
        v[int(b["page_table"][s, j // page]), h, j % page, e] = bad
        zeroed[int(b["page_table"][s, j // page]), h, j % page, e] = 0
    for j in range(prefix * page - 1, max(0, prefix * page - 60), -13):
        i = int(b["prefix_pages"][j // page])
        v[i, j % hk, j % page, j % d], zeroed[i, j % hk, j % page, j % d] = bad, 0
    ref, rl, spread = attention(q, k, zeroed, b, d ** -0.5)
    hit = torch.zeros(tokens, hq, d, dtype=torch.bool)
    for s, j, h, e in marks:
        for i in range(n_q[s]):
            if j <= kv[s] - n_q[s] + i:
                hit[int(b["q_start"][s]) + i, h * (hq // hk) : (h + 1) * (hq // hk), e] = True
    for j in range(prefix * page - 1, max(0, prefix * page - 60), -13):
        for s, n in enumerate(n_q):
            for i in range(n):
                if j <= prefix * page + kv[s] - n + i:
                    h = j % hk
                    hit[int(b["q_start"][s]) + i, h * (hq // hk) : (h + 1) * (hq // hk), j % d] = True
    lse = torch.empty(tokens, hq, device=DEV)
    out = g.paged_attention(ctx, q.to(DEV), k.to(DEV), v.to(DEV), *on_device(b), max_q=max_q, lse=lse,
                            prefix_pages=b["prefix_pages"].to(DEV) if prefix else None).cpu()
    done(ctx)
    assert hit.any() and not torch.isfinite(out[hit]).any()
    if not math.isnan(bad):
        assert torch.all((out[hit] == bad) | torch.isnan(out[hit]))   # (a weight that rounds to 0 makes NaN)
    check_attention(torch.where(hit, 0, out), lse.cpu(), torch.where(hit, 0, ref), rl, spread, "others")


def test_more_sequences_than_the_limit_are_refused(ctx):
    """By both calls, before anything is read (no array of that size exists here)."""
    cache = torch.zeros(2, 1, 16, 64, dtype=torch.float16, device=DEV)
    other = torch.zeros_like(cache)
    ints = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, y = (torch.zeros(2, 1, 64, dtype=torch.float16, device=DEV) for _ in range(2))
    c = bytes(serving.KvCache(cache.data_ptr(), other.data_ptr(), 2, 16, 1, 64, 1024, 1024, 64, serving.GEMM_F16))
    h, o = (bytes(serving.Heads(t.data_ptr(), 1, 64, 64)) for t in (x, y))
    r = bytes(serving.Rope(None, 0, None, None, 0.0, 1.0, 0))
    p, stream = ints.data_ptr(), torch.cuda.current_stream().cuda_stream
    of = lambda seqs, tokens: bytes(serving.KvBatch(seqs, tokens, 0, p, p, p, 1, 1, None, 0))
    assert g.lib().gemm_paged_attention_workspace(ctx.handle, c, of(2 ** 24, 0), 1) == 0
    assert g.lib().gemm_paged_attention_workspace(ctx.handle, c, of(2 ** 24 + 1, 0), 1) == g.GEMM_ERR_ARG
    assert g.lib().gemm_kv_append(ctx.handle, c, of(2 ** 24 + 1, 2), h, h, h, r, o, stream) == g.GEMM_ERR_ARG
    done(ctx)
