// Host check of the ranges that paged_attention_kernel cuts its work into: for one launch, every
// CTA's walk, one after the other, and that together they cover each block of each item once, in order.
//   schedule_walk tiles group kv_heads page_size prefix_pages keys seqs tile_tokens grid n:kv [n:kv ...]
// prints "ok units largest_head ctas" or what is wrong.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "paged_attention_kernel.cuh"

using namespace gb300;

template <class Cfg>
int check(PagedParams p, int grid)
{
    const int seqs = seq_count(p);
    auto sum = [&](int quantum, int64_t *largest) {
        int64_t total = 0;
        for (int s = 0; s < seqs; ++s) {
            const int64_t head = units_of_head<Cfg>(seq_items<Cfg>(p, s), quantum);
            *largest = head > *largest ? head : *largest;
            total += p.kv_heads * head;
        }
        return total;
    };
    // the closed form of a head's units against the sum over its tiles
    for (int quantum : {1, kPagedQuantum})
        for (int s = 0; s < seqs; ++s) {
            const SeqItems q = seq_items<Cfg>(p, s);
            int64_t units = 0;
            for (int t = 0; t < q.tiles; ++t)
                units += units_upto<Cfg>(q, quantum, min((t + 1) * q.step, q.n) - 1);
            if (units != units_of_head<Cfg>(q, quantum)) {
                printf("sequence %d, quantum %d: %lld units, not %lld\n", s, quantum, (long long)units_of_head<Cfg>(q, quantum),
                       (long long)units);
                return 1;
            }
        }
    int64_t largest = 0;
    int quantum = 1;
    Shares shares;
    shares.total = sum(1, &largest);
    if (Cfg::NT == 2 && shares.total < static_cast<int64_t>(kPagedCoarse) * grid) {
        quantum = kPagedQuantum;
        shares.total = sum(quantum, &largest);
    }
    shares.ctas = static_cast<int>(min(static_cast<int64_t>(grid), shares.total));
    // what comes next: sequence, head, tile, block
    int s = -1, head = 0, tile = 0, block = 0;
    SeqItems q = {};
    auto settle = [&] {   // on to the next tile that there is
        while (s < seqs && tile >= q.tiles) {
            tile = block = 0;
            if (s >= 0 && q.tiles > 0 && ++head < p.kv_heads)
                return;
            head = 0;
            if (++s < seqs)
                q = seq_items<Cfg>(p, s);
        }
    };
    settle();
    int open = -1;   // CTA that began the item which goes on, and the parts that it expects
    int parts = 0, seen = 0;
    for (int c = 0; c < shares.ctas; ++c) {
        const int64_t u0 = shares.begin(c);
        Walk w = {};
        int64_t before = 0, at = 0;
        for (int i = 0; i < seqs; ++i) {
            const SeqItems x = seq_items<Cfg>(p, i);
            const int64_t per_head = units_of_head<Cfg>(x, quantum), own = p.kv_heads * per_head;
            if (own > 0 && before <= u0 && u0 < before + own) {
                w.s = i;
                w.q = x;
                w.head = static_cast<int>((u0 - before) / per_head);
                at = u0 - before - w.head * per_head;
                w.unit = x.tiles > 1 ? 0 : static_cast<int>(at);
                break;
            }
            before += own;
        }
        w.quantum = quantum;
        w.left = shares.begin(c + 1) - u0;
        if (w.q.tiles > 1) {
            int found = 0;
            locate_tile<Cfg>(
                w.q, quantum, at, 0, 1,
                [](int64_t v, int64_t &ahead) {
                    ahead = 0;
                    return v;
                },
                [&](int t, int unit) {
                    w.tile = t;
                    w.unit = unit;
                    ++found;
                });
            if (found != 1) {
                printf("CTA %d: the tile of unit %lld was found %d times\n", c, (long long)at, found);
                return 1;
            }
        }
        Segment g;
        while (next_segment<Cfg>(p, w, g)) {
            const int want_s = p.keys == KEYS_BOTH ? s - 1 : s;
            const int first = tile * q.step, toks = min(q.step, q.n - first);
            const int blocks = blocks_upto<Cfg>(q, first + toks - 1);
            if (s >= seqs || g.s != want_s || g.head != head || g.tok0 != q.q0 + first || g.toks != toks || g.b0 != block ||
                g.b1 <= g.b0 || g.b1 > blocks || g.blocks != blocks) {
                printf("CTA %d: sequence %d head %d token %d blocks %d..%d of %d; expected %d %d %d from %d of %d\n", c, g.s, g.head,
                       g.tok0, g.b0, g.b1, g.blocks, want_s, head, q.q0 + first, block, blocks);
                return 1;
            }
            if (g.b0 == 0 && g.b1 < g.blocks) {   // as the softmax warps count the parts of an item
                open = c;
                parts = shares.owner(shares.begin(c + 1) - g.ahead + g.units - 1) - c + 1;
                seen = 1;
            } else if (g.b0 > 0) {
                ++seen;
                if (c != open + seen - 1 || (g.b1 == g.blocks && seen != parts)) {
                    printf("CTA %d: part %d of %d of an item begun in CTA %d\n", c, seen, parts, open);
                    return 1;
                }
            }
            block = g.b1;
            if (block == blocks) {
                ++tile;
                block = 0;
                settle();
            }
        }
    }
    if (s < seqs) {
        printf("sequence %d head %d tile %d block %d and what follows: of no CTA\n", s, head, tile, block);
        return 1;
    }
    printf("ok %lld %lld %d\n", (long long)shares.total, (long long)largest, shares.ctas);
    return 0;
}

int main(int argc, char **argv)
{
    if (argc < 11)
        return 2;
    PagedParams p = {};
    const int tiles = atoi(argv[1]);
    p.group = atoi(argv[2]);
    p.kv_heads = atoi(argv[3]);
    while ((1 << p.batch.page_shift) < atoi(argv[4]))
        ++p.batch.page_shift;
    p.batch.prefix_len = atoi(argv[5]) << p.batch.page_shift;
    p.keys = atoi(argv[6]);
    p.seqs = atoi(argv[7]);
    p.long_tokens = 128 / p.group;
    p.tile_tokens = atoi(argv[8]);
    std::vector<int> start(1, 0), lens;
    for (int i = 10; i < argc; ++i) {
        char *colon;
        start.push_back(start.back() + static_cast<int>(strtol(argv[i], &colon, 10)));
        lens.push_back(atoi(colon + 1));
    }
    p.batch.q_start = start.data();
    p.batch.kv_lens = lens.data();
    p.batch.num_seqs = static_cast<int>(lens.size());
    p.batch.num_tokens = start.back();
    p.batch.table_width = (2147482624 >> p.batch.page_shift) - atoi(argv[5]);
    return tiles == 1 ? check<PagedConfig<__half, 128, 1>>(p, atoi(argv[9])) : check<PagedConfig<__half, 128, 2>>(p, atoi(argv[9]));
}
