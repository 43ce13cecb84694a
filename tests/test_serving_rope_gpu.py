"""Norm and rotation of query and key heads, strided and into a paged cache, against 64 bits."""
import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from serving_ref import TYPES, batch, check_rope, rope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6


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


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype,tokens,hq,hk,d,rd", [
    ("float16", 1, 1, 1, 64, 64), ("bfloat16", 1, 32, 8, 128, 128), ("float16", 7, 5, 1, 128, 16),
    ("bfloat16", 33, 7, 7, 64, 48), ("float16", 130, 20, 4, 128, 80), ("bfloat16", 700, 64, 8, 128, 128),
    ("float16", 257, 3, 3, 64, 16), ("float16", 65, 17, 2, 128, 0)], ids=str)
def test_qk_rope_matches_64_bits(ctx, dtype, tokens, hq, hk, d, rd, norm, interleaved):
    t = TYPES[dtype]
    qkv = normal((tokens, (hq + 2 * hk) * d), tokens + hq, t)   # a packed projection
    qd = dev(qkv)
    cut = [hq * d, hk * d, hk * d]
    q, k, _ = qkv.split(cut, 1)
    qs, ks, _ = qd.split(cut, 1)
    q, k, qs, ks = q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d)), qs.unflatten(1, (hq, d)), ks.unflatten(1, (hk, d))
    wq, wk = (1 + 0.3 * normal((d,), 1, torch.float32)).to(t), (1 + 0.3 * normal((d,), 2, torch.float32)).to(t)
    wq, wk = (wq, wk) if norm else (None, None)
    table, scale = g.rope_table(rd, 10000.0, "yarn", 8.0, 4096) if rd else (None, 1.0)
    pos = torch.randint(0, 2 ** 31 - 1, (tokens,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    pos[: tokens // 2] = torch.arange(tokens // 2, dtype=torch.int32)
    qo, ko = g.qk_rope(ctx, qs, ks, dev(pos), dev(table), interleaved=interleaved, rope_scale=scale, q_norm=dev(wq),
                       k_norm=dev(wk), eps=EPS)
    done(ctx)
    for got, x, w, what in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        ref, mag = rope(x, w, pos, table, interleaved, scale, EPS)
        check_rope(got.cpu(), ref, mag, what)
    assert torch.equal(qd.cpu(), qkv)


def test_negative_positions_and_one_norm_only(ctx):
    t, d = torch.float16, 128
    q, k = normal((6, 4, d), 1, t), normal((6, 2, d), 2, t)
    w = normal((d,), 3, t)
    table, _ = g.rope_table(d)
    pos = torch.tensor([-1, -2 ** 31, 2 ** 31 - 1, 0, -77, 1], dtype=torch.int32)
    qo, ko = g.qk_rope(ctx, dev(q), dev(k), dev(pos), dev(table), k_norm=dev(w), eps=EPS)
    done(ctx)
    check_rope(qo.cpu(), *rope(q, None, pos, table, False, 1.0, EPS), "q")
    check_rope(ko.cpu(), *rope(k, w, pos, table, False, 1.0, EPS), "k")


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_inside_a_packed_projection(ctx, interleaved):
    t, tokens, hq, hk, d = torch.bfloat16, 50, 6, 2, 64
    qkv = normal((tokens, (hq + 2 * hk) * d), 5, t)
    w = normal((d,), 6, t)
    x = dev(qkv)

    def cut(y):
        return y[:, : hq * d].unflatten(1, (hq, d)), y[:, hq * d : (hq + hk) * d].unflatten(1, (hk, d))

    q, k = cut(x)
    table, _ = g.rope_table(32)
    pos = torch.arange(tokens, dtype=torch.int32) + 1000
    g.qk_rope(ctx, q, k, dev(pos), dev(table), interleaved=interleaved, q_norm=dev(w), eps=EPS, q_out=q, k_out=k)
    done(ctx)
    y = x.cpu()
    check_rope(cut(y)[0], *rope(cut(qkv)[0], w, pos, table, interleaved, 1.0, EPS), "q")
    check_rope(cut(y)[1], *rope(cut(qkv)[1], None, pos, table, interleaved, 1.0, EPS), "k")
    assert torch.equal(y[:, (hq + hk) * d :], qkv[:, (hq + hk) * d :])


def test_head_major_outputs_feed_the_contiguous_attention(ctx):
    t, s, h, d = torch.float16, 300, 4, 128
    x = normal((s, 3 * h * d), 9, t)
    q, k, v = (x[:, i * h * d : (i + 1) * h * d].unflatten(1, (h, d)) for i in range(3))
    table, _ = g.rope_table(d)
    pos = torch.arange(s, dtype=torch.int32)
    xd = dev(x)
    qd, kd, vd = (xd[:, i * h * d : (i + 1) * h * d].unflatten(1, (h, d)) for i in range(3))
    qo, ko = (torch.empty(h, s, d, dtype=t, device=DEV) for _ in range(2))
    g.qk_rope(ctx, qd, kd, dev(pos), dev(table), q_out=qo.transpose(0, 1), k_out=ko.transpose(0, 1))
    out = g.attention(ctx, qo, ko, vd.transpose(0, 1).contiguous(), causal=True)
    done(ctx)
    qr, _ = rope(q, None, pos, table, False, 1.0, EPS)
    kr, _ = rope(k, None, pos, table, False, 1.0, EPS)
    score = torch.einsum("shd,thd->hst", qr, kr) / d ** 0.5
    score = score.masked_fill(torch.ones(s, s, dtype=torch.bool).triu(1), float("-inf"))
    ref = torch.einsum("hst,thd->hsd", torch.softmax(score, -1), v.double())
    # q and k are rounded (2^-11 each, of scores up to about 5), then the attention's own 3e-3 + 4e-3 |ref|
    assert torch.all((out.cpu().double() - ref).abs() <= 1.2e-2 + 4e-3 * ref.abs())


N_Q = {"one": [1], "decode": [1] * 13, "ragged": [3, 0, 1, 130, 0, 17], "first_empty": [0, 0, 5], "many": [1, 2] * 150}


@pytest.mark.parametrize("by_rows", [False, True])
@pytest.mark.parametrize("dtype,hq,hk,d,rd,page,prefix", [("float16", 4, 2, 128, 128, 16, 0), ("bfloat16", 8, 1, 64, 32, 64, 3),
                                                          ("float16", 3, 3, 64, 64, 256, 0), ("bfloat16", 10, 5, 128, 0, 32, 1)],
                         ids=str)
@pytest.mark.parametrize("lens", list(N_Q))
def test_kv_append_matches_64_bits(ctx, lens, dtype, hq, hk, d, rd, page, prefix, by_rows):
    t, n_q = TYPES[dtype], N_Q[lens]
    kv = [n + (37 * i) % 300 for i, n in enumerate(n_q)]
    b = batch(n_q, kv, page, prefix_pages=prefix, seed=len(n_q))
    tokens = sum(n_q)
    spare = 5   # tokens behind the last sequence
    q, k, v = normal((tokens + spare, hq, d), 1, t), normal((tokens + spare, hk, d), 2, t), normal((tokens + spare, hk, d), 3, t)
    v[0, 0, 0] = float("nan")   # values are copied as they are
    shape = (b["pages"], page, hk, d) if by_rows else (b["pages"], hk, page, d)
    before = [normal(shape, 4 + i, t) for i in range(2)]
    caches = [dev(x) for x in before]
    views = [x.transpose(1, 2) if by_rows else x for x in caches]
    wq, wk = normal((d,), 7, t), normal((d,), 8, t)
    table = g.rope_table(rd)[0] if rd else None
    q_out = torch.full((tokens + spare, hq, d), 7.0, dtype=t, device=DEV)
    g.kv_append(ctx, dev(q), dev(k), dev(v), *views, dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]), dev(table),
                prefix_len=prefix * page, rope_scale=1.25, q_norm=dev(wq), k_norm=dev(wk), eps=EPS, q_out=q_out)
    done(ctx)
    want_k, want_v = (x.transpose(1, 2).clone() if by_rows else x.clone() for x in before)
    got_k, got_v = (x.cpu() for x in views)
    touched = torch.zeros(b["pages"], page, dtype=torch.bool)
    pos, page_of, row_of = [], [], []
    for s, n in enumerate(n_q):
        for i in range(n):
            place = kv[s] - n + i
            pos.append(prefix * page + place)
            page_of.append(int(b["page_table"][s, place // page]))
            row_of.append(place % page)
    pg, rw = torch.tensor(page_of), torch.tensor(row_of)
    touched[pg, rw] = True
    ref_q, mag_q = rope(q[:tokens], wq, pos, table, False, 1.25, EPS)
    check_rope(q_out[:tokens].cpu(), ref_q, mag_q, "q")
    assert torch.all(q_out[tokens:] == 7.0)
    ref_k, mag_k = rope(k[:tokens], wk, pos, table, False, 1.25, EPS)
    check_rope(got_k[pg, :, rw], ref_k, mag_k, "k")
    assert torch.equal(got_v[pg, :, rw].view(torch.int16), v[:tokens].view(torch.int16))
    keep = ~touched[:, None, :, None].expand_as(want_k)
    assert torch.equal(got_k[keep], want_k[keep]) and torch.equal(got_v[keep], want_v[keep])


def test_kv_append_without_queries_and_in_place(ctx):
    t, hk, d, page = torch.float16, 2, 128, 16
    b = batch([2, 3], [20, 3], page)
    k, v, q = normal((5, hk, d), 1, t), normal((5, hk, d), 2, t), normal((5, 4, d), 3, t)
    kc, vc = (torch.zeros(b["pages"], hk, page, d, dtype=t, device=DEV) for _ in range(2))
    table, _ = g.rope_table(d)
    args = (dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]), dev(table))
    assert g.kv_append(ctx, None, dev(k), dev(v), kc, vc, *args) is None
    one = kc.clone()
    qd = dev(q)
    assert g.kv_append(ctx, qd, dev(k), dev(v), kc, vc, *args, q_out=qd) is qd
    done(ctx)
    assert torch.equal(one, kc)
    check_rope(qd.cpu(), *rope(q, None, [18, 19, 0, 1, 2], table, False, 1.0, EPS), "q")


def test_one_cache_tensor_holding_keys_and_values(ctx):
    """Keys and values of a page side by side in one tensor: [pages, 2, kv_heads, page_size, head_dim]."""
    t, hk, d, page = torch.bfloat16, 3, 64, 32
    b = batch([4], [50], page)
    both = torch.zeros(b["pages"], 2, hk, page, d, dtype=t, device=DEV)
    k, v = normal((4, hk, d), 1, t), normal((4, hk, d), 2, t)
    g.kv_append(ctx, None, dev(k), dev(v), both[:, 0], both[:, 1], dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"]))
    done(ctx)
    got = both.cpu()
    for i in range(4):
        place = 46 + i
        pg = int(b["page_table"][0, place // page])
        assert torch.equal(got[pg, 0, :, place % page], k[i]) and torch.equal(got[pg, 1, :, place % page], v[i])
    assert int((got != 0).any(-1).sum()) == 4 * 2 * hk


def test_captured_append_follows_new_lengths(ctx):
    t, hk, d, page, n = torch.float16, 2, 128, 16, 3
    b = batch([1] * n, [40] * n, page)
    k, v = normal((n, hk, d), 1, t), normal((n, hk, d), 2, t)
    kd, vd = dev(k), dev(v)
    kc, vc = (torch.zeros(b["pages"], hk, page, d, dtype=t, device=DEV) for _ in range(2))
    q_start, kv, pt = dev(b["q_start"]), dev(b["kv_lens"]), dev(b["page_table"])
    kv.fill_(1)
    table = g.rope_table(d)[0]
    td = dev(table)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        g.kv_append(ctx, None, kd, vd, kc, vc, q_start, kv, pt, td)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            g.kv_append(ctx, None, kd, vd, kc, vc, q_start, kv, pt, td)
    torch.cuda.current_stream().wait_stream(stream)
    for step in (5, 17, 40):
        kv.fill_(step)
        graph.replay()
        done(ctx)
        for s in range(n):
            pg = int(b["page_table"][s, (step - 1) // page])
            got = kc[pg, :, (step - 1) % page].cpu()
            check_rope(got[None], *rope(k[s : s + 1], None, [step - 1], table, False, 1.0, EPS), step)


@pytest.mark.parametrize("what", ["page", "page_negative", "kv_long", "kv_negative", "kv_short", "q_start"])
def test_bad_batches_touch_nothing_and_are_reported(ctx, what):
    """Indexes out of range are left out by the kernel's own checks (tokens of other sequences
    are written as always)."""
    t, hk, d, page = torch.float16, 2, 64, 16
    b = batch([2, 2], [10, 20], page)
    pt, kv, qs = b["page_table"].clone(), b["kv_lens"].clone(), b["q_start"].clone()
    if what == "page":
        pt[1, 1] = b["pages"]
    elif what == "page_negative":
        pt[1, 1] = -5
    elif what == "kv_long":
        kv[1] = 3 * page
    elif what == "kv_negative":
        kv[1] = -2 ** 31
    elif what == "kv_short":
        kv[1] = 0
    else:
        qs[2] = 100
    k, v = normal((4, hk, d), 1, t), normal((4, hk, d), 2, t)
    kc, vc = (torch.zeros(b["pages"], hk, page, d, dtype=t, device=DEV) for _ in range(2))
    g.kv_append(ctx, None, dev(k), dev(v), kc, vc, dev(qs), dev(kv), dev(pt))
    torch.cuda.synchronize()
    assert g.gemm_last_device_error(ctx) == (g.GEMM_ERR_INDEX, 8)
    assert g.gemm_last_device_error(ctx) == (g.GEMM_OK, 0)
    got = kc.cpu()
    assert torch.equal(got[int(b["page_table"][0, 0]), :, 8:10].transpose(0, 1), k[:2])
