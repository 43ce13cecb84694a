"""The serving operators where numbers or calls are out of the ordinary: keys and values that are not
finite, scores of minus infinity only, a key far ahead of a long context, scales near zero, outputs
on another stream, bad lengths of sequences without tokens."""
import math

import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from tensor_core_gemm_tcgen05_gb300 import serving
from serving_ref import TYPES, attention, batch, check_attention, half_step, keys_of, tiny

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


def run(ctx, b, q, k, v, max_q=None, scale=None):
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    pages = None if b["prefix_pages"] is None else b["prefix_pages"].to(DEV)
    out = g.paged_attention(ctx, q.to(DEV), k.to(DEV), v.to(DEV), b["q_start"].to(DEV), b["kv_lens"].to(DEV), b["page_table"].to(DEV),
                            max_q=max_q, prefix_pages=pages, scale=scale, lse=lse)
    done(ctx)
    return out.cpu(), lse.cpu()


def by_rows(q, k, v, b, scale):
    """(out, lse, spread) in 64 bits, each row over the keys that it sees and no others, with what
    infinities and NaN among them make of it: 0/0 where no weight is left, 0 x inf, inf - inf."""
    tokens, hq, d = q.shape
    grp = hq // k.shape[1]
    out, spread = (torch.zeros(tokens, hq, d, dtype=torch.float64) for _ in range(2))
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64)
    for s, n in enumerate(b["n_q"]):
        ks, vs = (keys_of(x, b, s).double() for x in (k, v))
        for i in range(n):
            t, seen = int(b["q_start"][s]) + i, len(ks) - n + i + 1
            if seen <= 0:
                continue
            for h in range(hq):
                # the product of each pair, so that a matrix product's order plays no part
                score = (ks[:seen, h // grp] * q[t, h].double()).sum(-1) * scale
                p = torch.softmax(score, 0)[:, None]
                out[t, h], spread[t, h] = (p * vs[:seen, h // grp]).sum(0), (p * vs[:seen, h // grp].abs()).sum(0)
                lse[t, h] = torch.logsumexp(score, 0)
    return out, lse, spread


def check_any(out, lse, ref, ref_lse, spread, what):
    """Finite results within check_attention's bounds, NaN where the definition has it, infinities the
    same or NaN (a weight that rounds to 0 times one)."""
    fine = torch.isfinite(ref)
    got = out.double()
    wrong = torch.where(fine, ~torch.isfinite(got), torch.where(torch.isnan(ref), ~torch.isnan(got), (got != ref) & ~torch.isnan(got)))
    assert not wrong.any(), (what, int(wrong.sum()), wrong.nonzero()[:4].tolist(), ref[wrong][:4], got[wrong][:4])
    # (rows whose lse is finite or that see no key; the log of a sum with an infinite or NaN score is not a number either way)
    num = torch.isfinite(ref_lse) | (ref_lse == -math.inf)
    assert not torch.isfinite(lse[~num]).any(), what
    assert torch.equal(lse[ref_lse == -math.inf].double(), ref_lse[ref_lse == -math.inf]), what
    err = (lse.double() - ref_lse)[torch.isfinite(ref_lse)].abs() / (2.0 ** -16 + 2.0 ** -22 * ref_lse[torch.isfinite(ref_lse)].abs())
    assert err.numel() == 0 or float(err.max()) <= 1.0, what
    bound = half_step(out.dtype) * ref.abs() * (1 + 2.0 ** -7) + (half_step(out.dtype) + 2.0 ** -16) * spread + tiny(out.dtype)
    err = ((got - ref).abs() / bound)[fine]
    assert err.numel() == 0 or float(err.max()) <= 1.0, (what, float(err.max()))


def spots(b, hk, d, count, seed, late):
    """Random (sequence, own key, head, dim); `late`: among the new keys."""
    gen = torch.Generator().manual_seed(seed)
    pick = lambda n: int(torch.randint(0, n, (1,), generator=gen))
    at = []
    for s, n in enumerate(b["kv"]):
        for _ in range(count if n else 0):
            j = n - 1 - pick(min(n, max(1, b["n_q"][s]))) if late else pick(n)
            at.append((s, j, pick(hk), pick(d)))
    return at


def put(x, b, at, value):
    for s, j, h, e in at:
        x[int(b["page_table"][s, j // b["page_size"]]), h, j % b["page_size"], e] = value



@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("n_q,kv,hq,hk,d,page,prefix,max_q", [
    ([4] * 160, [30 + i % 9 for i in range(160)], 8, 4, 64, 16, 0, 4),       # several items to a CTA
    ([4] * 160, [30 + i % 9 for i in range(160)], 4, 4, 128, 32, 0, None),
    ([70, 3, 130], [300, 67, 131], 4, 2, 64, 64, 0, None),
    ([3, 5], [700, 5], 4, 2, 128, 16, 0, 5),
    ([6] * 20, [20] * 20, 4, 1, 64, 16, 9, 6),
    ([150], [150], 2, 1, 128, 16, 3, None)], ids=lambda x: str(x)[:20])
def test_keys_and_values_that_are_not_finite(ctx, n_q, kv, hq, hk, d, page, prefix, max_q, bad):
    """In keys (the first of a sequence, which all rows see, and others), in late values that earlier new
    tokens do not see, and both at once."""
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=8)
    q = normal((sum(n_q), hq, d), 1)
    first = [(s, 0, s % hk, s % d) for s in range(0, len(kv), 2) if kv[s]]
    late = spots(b, hk, d, 2, 3, late=True)
    for what, in_k, in_v in (("keys", first + spots(b, hk, d, 1, 4, late=False)[::3], []), ("late keys", spots(b, hk, d, 1, 5, late=True), []),
                             ("values", [], late), ("both", first, late), ("late both", late[::2], late[1::2])):
        k, v = normal((b["pages"], hk, page, d), 2), normal((b["pages"], hk, page, d), 3)
        put(k, b, in_k, bad)
        put(v, b, in_v, bad)
        check_any(*run(ctx, b, q, k, v, max_q=max_q), *by_rows(q, k, v, b, d ** -0.5), what)


@pytest.mark.parametrize("n_q,kv,hq,hk,d,page,prefix,max_q", [
    ([1, 3, 1], [70, 5, 1], 4, 2, 64, 16, 0, 3), ([1, 1], [3000, 90], 4, 2, 128, 16, 0, 1), ([200, 40], [200, 60], 4, 2, 64, 16, 0, None),
    ([1] * 12, [30] * 12, 4, 2, 64, 16, 8, 1), ([150, 2, 1], [150, 5, 9], 4, 2, 128, 16, 2, None), ([5, 40], [2, 20], 4, 1, 64, 16, 0, 40)],
    ids=lambda x: str(x)[:20])
def test_rows_whose_scores_are_all_minus_infinity(ctx, n_q, kv, hq, hk, d, page, prefix, max_q):
    """No weight is left and a key is seen: 0/0, not the zeros of a row that sees none. One such key among
    others only loses its weight; a whole such prefix leaves the own keys theirs."""
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=8)
    q = normal((sum(n_q), hq, d), 1)
    q[..., 3] = q[..., 3].abs() + 0.5   # (so that -inf in that dim is -inf in the score)
    v = normal((b["pages"], hk, page, d), 3)
    plain = normal((b["pages"], hk, page, d), 2)
    every = [(s, j, h, 3) for s in range(len(kv)) for j in range(kv[s]) for h in range(hk)]
    for what, own, pre in (("all", every, True), ("one head", [x for x in every if x[2] == 0], False), ("the first key", [x for x in every if x[1] == 0], False),
                           ("all but the last", [x for x in every if x[1] < kv[x[0]] - 1], True), ("the prefix", [], True)):
        k = plain.clone()
        put(k, b, own, -math.inf)
        if pre and prefix:
            k[b["prefix_pages"].long(), ..., 3] = -math.inf
        check_any(*run(ctx, b, q, k, v, max_q=max_q), *by_rows(q, k, v, b, d ** -0.5), what)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ahead", [0.0, 10.0, 14.0, 16.0, 17.4])
@pytest.mark.parametrize("n_q,seqs,sink", [(1, 200, 0), (1, 200, 20000), (130, 50, 0)])
def test_a_key_far_ahead_of_a_long_context(ctx, n_q, seqs, sink, ahead, dtype):
    """One key whose value is zero and whose score is ahead of 32767 equal ones, in as many sequences (of the
    same pages) as leave most items to one CTA: the output is what the many small weights leave. Each is
    off by half a step of the type at most, or by half of FP16's smallest step 2^-24, the largest weight
    being 2^11 or more; what check_attention counts besides is the same."""
    t, hk, d, page, n = TYPES[dtype], 8, 64, 1024, 32768
    b = batch([n_q], [n], page, seed=1)
    k = torch.zeros(b["pages"], hk, page, d, dtype=t)
    v = (torch.rand(b["pages"], 1, page, d, generator=torch.Generator().manual_seed(2)) + 0.5).to(t).repeat(1, hk, 1, 1)
    put(k, b, [(0, sink, h, 0) for h in range(hk)], ahead)
    v[int(b["page_table"][0, sink // page]), :, sink % page] = 0
    q = torch.zeros(seqs * n_q, 2 * hk, d, dtype=t)
    q[..., 0] = 1
    x = float(k.max())   # (rounded to the type)
    many = dict(b, q_start=torch.arange(0, seqs * n_q + 1, n_q, dtype=torch.int32), kv_lens=b["kv_lens"].repeat(seqs),
                page_table=b["page_table"].repeat(seqs, 1))
    out, lse = run(ctx, many, q, k, v, max_q=n_q, scale=1.0)
    values = keys_of(v, b, 0)[:, 0].double().cumsum(0)
    seen = torch.arange(n - n_q + 1, n + 1)
    total = math.exp(x) + (seen - 1).double()
    ref = (values[seen - 1] / total[:, None])[:, None]
    step = half_step(t)
    bound = step * ref * (1 + 2.0 ** -7) + (step + 2.0 ** -16) * ref
    if t == torch.float16:
        bound = bound + 2.0 ** -36 * math.exp(x) * ref
    got = out.double().view(seqs, n_q, 2 * hk, d)
    assert float(((got - ref).abs() / bound).max()) <= 1.0, float(((got - ref).abs() / ref).max())
    err = (lse.double().view(seqs, n_q, 2 * hk) - total.log()[:, None]).abs()
    # (the sum of exponentials grows block by block of 64 keys, n / 64 additions in FP32, each off by half a step
    # of a sum that hardly changes: at most 2^-24 of it, always the same way where the blocks are equal)
    assert float((err / (2.0 ** -16 + n / 64 * 2.0 ** -24 + 2.0 ** -22 * total.log()[:, None])).max()) <= 1.0


@pytest.mark.parametrize("scale", [0.0, 1e-39, -1e-39, 8.4e-39, -8.4e-39, 1e-38, -3e-38, -0.0], ids=str)
@pytest.mark.parametrize("n_q,kv", [([1, 4], [300, 70]), ([150], [150])], ids=str)
def test_scales_near_zero(ctx, n_q, kv, scale):
    """Scores up to 1e38, as bfloat16 queries and keys of 1e19 have them: scale 0 is the mean, and the
    smallest scales keep their size and sign (scale log2(e) below 2^-126 has 2^-149 as its step: with scores
    of 1e38 an error of 2^-23.8 in the exponent)."""
    b = batch(n_q, kv, 16, seed=3)
    q, k, v = (torch.zeros(s, dtype=torch.bfloat16) for s in ((sum(n_q), 4, 64), (b["pages"], 2, 16, 64), (b["pages"], 2, 16, 64)))
    q[..., 5] = 1e19
    k[..., 5] = normal(k.shape[:3], 1, torch.float32).clamp(-3, 3) * 3e18
    v.copy_(normal(v.shape, 2, torch.float32))
    ref = attention(q, k, v, b, scale)
    check_attention(*run(ctx, b, q, k, v, scale=scale), *ref, scale)


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_scales_that_leave_the_range_are_refused(ctx, scale):
    b = batch([1], [20], 16)
    q, k, v = normal((1, 2, 64), 1), normal((b["pages"], 1, 16, 64), 2), normal((b["pages"], 1, 16, 64), 3)
    with pytest.raises(g.GemmError) as e:
        run(ctx, b, q, k, v, scale=scale)
    assert e.value.status == g.GEMM_ERR_ARG
    done(ctx)


@pytest.mark.parametrize("call", ["qk_rope", "kv_append", "paged_attention"])
def test_outputs_for_another_stream_leave_freed_memory_alone(ctx, call):
    """A block that was freed on the current stream while queued work there still reads it must not become the
    output of a call on another stream."""
    n, hq, d = 4099, 8, 128
    b = batch([n], [n], 64, seed=1)
    q, k = normal((n, hq, d), 1).to(DEV), normal((n, hq, d), 2).to(DEV)
    kd, vd = (normal((b["pages"], hq, 64, d), 3 + i).to(DEV) for i in range(2))
    args = tuple(b[x].to(DEV) for x in ("q_start", "kv_lens", "page_table"))
    table, pos = g.rope_table(d)[0].to(DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    lse, copy = torch.empty(n, hq, device=DEV), torch.zeros(n, hq, d, dtype=torch.float16, device=DEV)
    ws = torch.empty(g.paged_attention_workspace(ctx, q, kd, vd, *args), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()

    def calls(stream):
        if call == "qk_rope":
            return g.qk_rope(ctx, q, k, pos, table, stream=stream)
        if call == "kv_append":
            return (g.kv_append(ctx, q, k, k, kd, vd, *args, table, stream=stream),)
        return (g.paged_attention(ctx, q, kd, vd, *args, lse=lse, workspace=ws, stream=stream),)

    want = [x.clone() for x in calls(None)]
    torch.cuda.synchronize()
    main = torch.cuda.default_stream()
    for current, stream in ((main, side), (main, side.cuda_stream), (side, main), (side, 0)):
        with torch.cuda.stream(current):
            old = [torch.full((n, hq, d), 3.0, dtype=torch.float16, device=DEV) for _ in want]
            torch.cuda.synchronize()
            torch.cuda._sleep(200_000_000)   # (about 0.1 s)
            for x in old:
                copy.add_(x)
            del old, x
            outs = calls(stream)
            torch.cuda.synchronize()
            assert torch.all(copy == 3.0 * len(want)), "a block still in use became the output"
            copy.zero_()
            for x, y in zip(outs, want):
                assert torch.equal(x, y)
            del outs, x, y
    done(ctx)


@pytest.mark.parametrize("what", ["kv_negative", "kv_long", "q_start_steps_back", "q_start_negative", "q_start_far"])
def test_bad_lengths_of_sequences_without_tokens_are_reported(ctx, what):
    """By gemm_kv_append as by attention, whether a token's search comes past them or not."""
    hk, d, page, n = 2, 64, 16, 300
    n_q = [i % 2 for i in range(n)]
    b = batch(n_q, [20] * n, page, seed=2)
    starts, lens = b["q_start"].clone(), b["kv_lens"].clone()
    if what == "kv_negative":
        lens[100] = -1
    elif what == "kv_long":
        lens[298] = b["page_table"].shape[1] * page + 1
    elif what == "q_start_steps_back":
        starts[101] -= 1   # (sequence 100, which has none; 101 then has one token more)
    elif what == "q_start_negative":
        starts[0] = -4
    else:
        starts[300] = 2 ** 31 - 1
    tokens = sum(n_q)
    q, k, v = (normal((tokens, h, d), i).to(DEV) for i, h in enumerate((4, hk, hk)))
    kd, vd = (torch.zeros(b["pages"], hk, page, d, dtype=torch.float16, device=DEV) for _ in range(2))
    args = (starts.to(DEV), lens.to(DEV), b["page_table"].to(DEV))
    g.kv_append(ctx, q, k, v, kd, vd, *args)
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_ERR_INDEX, 8)
    for s in range(1, 99, 2):   # sequences that nothing is wrong with
        assert torch.equal(vd[int(b["page_table"][s, 1]), :, 3], v[int(b["q_start"][s])])
    g.kv_append(ctx, q, k, v, kd, vd, *(b[x].to(DEV) for x in ("q_start", "kv_lens", "page_table")))
    done(ctx)


def test_join_after_a_timeout_reads_the_parts_only(ctx):
    """CTAs that give up leave the tokens' entries as the workspace had them: here such as would lead in front
    of the first token of a part, in a batch of fewer tokens than a tile takes."""
    n, hq, hk, d, page, prefix = 6, 8, 2, 64, 16, 30
    b = batch([1] * n, [20] * n, page, prefix_pages=prefix, seed=1)
    q, k, v = normal((n, hq, d), 1), normal((b["pages"], hk, page, d), 2), normal((b["pages"], hk, page, d), 3)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    args, pages = (b["q_start"].to(DEV), b["kv_lens"].to(DEV), b["page_table"].to(DEV)), b["prefix_pages"].to(DEV)
    ws = torch.empty(g.paged_attention_workspace(ctx, qd, kd, vd, *args, max_q=1, prefix_pages=pages), dtype=torch.uint8, device=DEV)
    lse = torch.empty(n, hq, device=DEV)
    g.gemm_set_timeout_ns(ctx, 20 * 10 ** 6)
    g.gemm_set_debug(ctx, g.GEMM_DEBUG_WITHHOLD_FIRST_LOAD)
    try:
        for first in (-20, -31, 0, 2 ** 31 - 1):
            ws.view(torch.int32).copy_(torch.tensor([0, 2, first, 0], dtype=torch.int32).repeat(ws.numel() // 16))
            g.paged_attention(ctx, qd, kd, vd, *args, max_q=1, prefix_pages=pages, lse=lse, workspace=ws)
            torch.cuda.synchronize()
            assert g.gemm_last_device_error(ctx)[0] == g.GEMM_ERR_TIMEOUT
    finally:
        g.gemm_set_debug(ctx, g.GEMM_DEBUG_NONE)
        g.gemm_set_timeout_ns(ctx, 2 * 10 ** 9)
    out = g.paged_attention(ctx, qd, kd, vd, *args, max_q=1, prefix_pages=pages, lse=lse, workspace=ws)
    done(ctx)
    check_attention(out.cpu(), lse.cpu(), *attention(q, k, v, b, d ** -0.5), "after")


def test_more_tokens_than_the_limit_are_refused(ctx):
    """By both calls, before anything is read (no array of that size exists here)."""
    cache = torch.zeros(2, 2, 1, 16, 64, dtype=torch.float16, device=DEV)
    c = bytes(serving.KvCache(cache[0].data_ptr(), cache[1].data_ptr(), 2, 16, 1, 64, 1024, 1024, 64, serving.GEMM_F16))
    of = lambda tokens: bytes(serving.KvBatch(0, tokens, 0, None, None, None, 1, 1, None, 0))
    h = bytes(serving.Heads(None, 0, 64, 64))
    k = bytes(serving.Heads(cache.data_ptr(), 1, 0, 0))
    r = bytes(serving.Rope(None, 0, None, None, 0.0, 1.0, 0))
    stream = torch.cuda.current_stream().cuda_stream
    for tokens, want in ((2 ** 31 - 1024, g.GEMM_OK), (2 ** 31 - 1023, g.GEMM_ERR_ARG), (2 ** 31 - 1, g.GEMM_ERR_ARG)):
        assert g.lib().gemm_paged_attention_workspace(ctx.handle, c, of(tokens), 1) == want
        assert g.lib().gemm_kv_append(ctx.handle, c, of(tokens), h, k, k, r, h, stream) == want
    done(ctx)


@pytest.mark.parametrize("slots,every,n,kv,prefix", [(3000, 61, 1, 40, 20), (3000, 700, 3, 9, 2), (5000, 2, 1, 5, 3), (700, 699, 2, 1, 4)], ids=str)
def test_prefix_of_a_padded_batch(ctx, slots, every, n, kv, prefix):
    """Tokens with many empty sequences before, between and behind them."""
    n_q = [n if i % every == every - 1 else 0 for i in range(slots)]
    b = batch(n_q, [kv if x else 0 for x in n_q], 16, prefix_pages=prefix, seed=4)
    q, k, v = normal((sum(n_q), 4, 64), 1), normal((b["pages"], 1, 16, 64), 2), normal((b["pages"], 1, 16, 64), 3)
    check_attention(*run(ctx, b, q, k, v, max_q=n), *attention(q, k, v, b, 0.125), "padded")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("top", [1e2, 4e3, 6e3, 1e5, 3e7, 2e8, 1e9, 3e10], ids=str)
@pytest.mark.parametrize("n_q,kv,prefix,scale", [([1, 3], [70, 300], 0, 1.0), ([150, 40], [150, 700], 0, 1.0), ([1] * 9, [50] * 9, 6, 0.7),
                                                 ([1], [9000], 0, -0.3), ([200], [900], 0, -0.9)], ids=lambda x: str(x)[:12])
def test_scores_of_any_size(ctx, n_q, kv, prefix, scale, top, dtype):
    """Scores whose FP32 steps are larger than the exponents of the type's probabilities: keys of the largest
    score share the weight (some in each sequence, so in several blocks, tiles and parts), the others, a tenth
    behind at least, have e^-10 of it or less. Queries of a power of two and keys of 64 equal values: FP32 holds
    the scores exactly."""
    t, page, d, hk = TYPES[dtype], 16, 64, 2
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=3)
    gen = torch.Generator().manual_seed(4)
    a = 2.0 ** math.floor(math.log2((top / abs(scale) / d) ** 0.5))
    most = top / abs(scale) / d / a
    x = (torch.rand(b["pages"], hk, page, 1, generator=gen) * 1.9 - 1) * most
    x[torch.rand(x.shape, generator=gen) < 0.02] = most
    q, k = torch.full((sum(n_q), 4, d), math.copysign(a, scale), dtype=t), x.to(t).repeat(1, 1, 1, d)
    v = normal(k.shape, 5, torch.float32).to(t)
    assert torch.isfinite(k).all() and torch.isfinite(q).all()
    check_attention(*run(ctx, b, q, k, v, scale=scale), *attention(q, k, v, b, scale), top)


@pytest.mark.parametrize("n_q,kv,hq,hk,d,page,prefix,max_q", [
    ([1] * 12, [1] * 12, 4, 2, 64, 16, 8, 1), ([1, 1], [3000, 90], 4, 2, 128, 16, 0, 1), ([3, 40], [70, 300], 4, 2, 64, 16, 0, 40),
    ([150, 2, 1], [150, 5, 9], 4, 2, 128, 16, 2, None), ([6] * 20, [9] * 20, 4, 1, 64, 16, 9, 6)], ids=lambda x: str(x)[:20])
def test_values_that_are_not_finite_of_keys_without_weight(ctx, n_q, kv, hq, hk, d, page, prefix, max_q):
    """A weight of 0 times an infinite value is NaN for the rows that see the key, wherever the keys are cut into
    parts, and nothing for the others."""
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=8)
    q = normal((sum(n_q), hq, d), 1)
    q[..., 3] = q[..., 3].abs() + 0.5
    for what, at in (("last", [(s, n - 1, s % hk, 3) for s, n in enumerate(kv)]), ("new", spots(b, hk, 1, 3, 5, late=True)),
                     ("late half", [(s, j, h, 3) for s, n in enumerate(kv) for j in range(n // 2, n) for h in range(hk)])):
        k, v = normal((b["pages"], hk, page, d), 2), normal((b["pages"], hk, page, d), 3)
        put(k, b, [(s, j, h, 3) for s, j, h, _ in at], -math.inf)
        put(v, b, [(s, j, h, (5 * j + s) % d) for s, j, h, _ in at], math.inf)
        check_any(*run(ctx, b, q, k, v, max_q=max_q), *by_rows(q, k, v, b, d ** -0.5), what)
