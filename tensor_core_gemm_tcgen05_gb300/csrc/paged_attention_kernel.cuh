// Attention of a ragged batch's new queries over a paged key/value cache (gemm_serving.h):
//
//     out[t][h] = sum_j p_j V[j][h'] / sum_j p_j,   p_j = 2^(s_j - m),  s_j = scale log2(e) q[t][h] . K[j][h']
//
// over the keys j at positions up to the token's own, in one pass over the keys with a running
// maximum m and sum l per row (FP32), on the fifth-generation tensor cores.
//
//  * Rows. The G query heads of a key head and consecutive tokens of a sequence are the rows of
//    one 128-row tile (row = token * G + head, 128 / G tokens), so a key block is read once for
//    all of them; one TMA box (64 dims x G heads x tokens) loads a tile from any strides. A
//    decoding token fills G rows and leaves the others idle: the tensor work of a block (two
//    128-row products) still takes less time than reading it (64 keys: 1024 clocks of two
//    products against about 1400 at an SM's share of HBM).
//  * Keys. A block of BKV keys is gathered by one TMA box per page (and 64 dims) at the page
//    table's page number; pages past the last key, and numbers out of range, are addressed one
//    past the last page, which TMA fills with zeros. Rows of a page past the last key hold
//    anything (NaN too): their scores are masked, and their rows of V are zeroed in shared
//    memory before the product (0 x NaN would be NaN).
//  * Work. An item is (sequence, key head, tile or pair of tiles), its cost its key blocks. The
//    blocks of all items in order (units) are cut into one equal range per CTA (every CTA adds
//    up the lengths itself, on the device, so a captured graph follows them): no CTA waits for
//    another, and long and short sequences balance. An item cut by a range boundary leaves one
//    part per CTA, (m, l, O) in FP32 in the workspace, joined by paged_combine_kernel; an item
//    inside one range is finished here.
//  * Two forms. NT = 1: one tile, blocks of 64 keys, two score buffers, two CTAs per SM (for
//    few rows: bound by HBM; one CTA's latencies overlap the other's). NT = 2: two tiles share
//    each block of 128 keys, one CTA per SM (for many rows: bound by the tensor cores; one
//    tile's softmax runs during the other's products).
//  * Warps: four softmax warps per tile, a row per thread, an MMA issuer and a producer (TMA), as
//    in attention_fwd_kernel. Every wait is bounded.
#pragma once

#include <type_traits>

#include "serving_common.cuh"

namespace gb300 {

// Which keys a launch covers.
enum : int {
    KEYS_ALL = 0,     // the prefix (if any), then the sequence's own
    KEYS_OWN = 1,     // the sequence's own (the prefix is another launch's)
    KEYS_PREFIX = 2,  // the prefix, for the tokens of all sequences together
    KEYS_BOTH = 3,    // the items of KEYS_PREFIX, then those of KEYS_OWN
};
// Which sequences a launch takes, by their new tokens against a tile's.
enum : int { SEQS_ALL = 0, SEQS_SHORT = 1, SEQS_LONG = 2 };

// Parts of the workspace of one launch: what a CTA leaves of items that are cut.
struct PartsView {
    float *o;        // [2 * CTAs][tiles * rows][D]: part 0: began in an earlier CTA; 1: goes on in the next
    float2 *ml;      // [2 * CTAs][tiles * rows] (m, l)
    int rows;        // rows kept per tile
    int tiles;
};

// Where the parts of an item are. For each CTA, of the item that goes on past its range (its part
// 1): {first token, tokens, key head, parts}, parts = 0 if there is none. For each token and key
// head, when the prefix is a launch of its own: {CTA of the first part, parts (1: whole, in the
// row tables), the item's first token, launch}.
using PartInfo = int4;

struct PagedParams {
    BatchView batch;
    const int *prefix_pages;
    int n_prefix_pages;
    int kv_heads, group;                // G: query heads per key head
    int tile_tokens, long_tokens;       // tokens per tile of this launch; what a full tile takes, 128 / G:
                                        // the tile of prefix items
    int q_rows, q_bufs;                 // NT = 1: rows of a query buffer (whole groups of 8), buffers
    int busy_warps;                     // softmax warps of a tile that can have rows (the others leave at once)
    int keys, seqs;                     // KEYS_*, SEQS_*
    int launch;                         // index for the tokens' PartInfo
    float scale_log2;                   // scale * log2(e)
    void *out;
    int64_t out_token, out_head;
    float *lse;
    int64_t lse_token;
    PartsView parts;
    PartInfo *cuts;                     // [CTAs]; KEYS_ALL only
    // not KEYS_ALL, of own [0] and of prefix keys [1]:
    PartInfo *info[2];                  // [num_tokens][kv_heads]
    float *row_o[2];                    // whole items, [num_tokens][heads][D]
    float2 *row_ml[2];
    // what repair_stretches reads: the operands as the tensor maps have them, strides in elements
    const void *q, *k, *v;
    int64_t q_token, q_head, page_stride, head_stride, row_stride;
    uint32_t *err;
    uint64_t timeout_ns;
    int debug;                          // DEBUG_WITHHOLD_FIRST_LOAD
};

template <typename T, int D_, int NT_>
struct PagedConfig {
    using Type = T;
    static constexpr int D = D_;
    static constexpr int NT = NT_;                  // query tiles per item
    static constexpr int BQ = 128;                  // rows per tile (= TMEM lanes)
    static constexpr int BKV = NT == 1 ? 64 : 128;  // keys per block
    static constexpr int ATOMS = D / 64;            // 128-byte-swizzled atoms of 64 dims
    static constexpr int Q_ATOM = BQ * 128, Q_TILE = ATOMS * Q_ATOM;
    static constexpr int KV_ATOM = BKV * 128, KV_TILE = ATOMS * KV_ATOM;
    // ring of K and V tiles (K0 V0 K1 V1 ...): what fits beside Q in half of (NT = 1) or all of
    // an SM's shared memory
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int Q_OFF = 0, RING_OFF = NT * Q_TILE;
    // NT = 2: 32 rows x 128 bytes for each softmax warp, through which results are written
    static constexpr int STAGE_WARP = 32 * 128, STAGE_OFF = RING_OFF + STAGES * KV_TILE;
    static constexpr int BAR_OFF = STAGE_OFF + (NT == 2 ? 8 * STAGE_WARP : 0);
    // q_full[], q_empty[], drain, full[], empty[], s_full and pv_done (NT = 2: of the first tile),
    // then NT = 1: p_full[block mod 2]; NT = 2: p_half[tile], p_full[tile]
    static constexpr int Q_BUFS = NT == 1 ? 4 : 1;   // at most
    static constexpr int NUM_BARS = 2 * Q_BUFS + 1 + 2 * STAGES + 2 + 2 * NT;
    // what beginning and ending an item costs, in blocks
    static constexpr int ITEM_COST = 2;
    // Probabilities are kept as P = 2^(s - m), m = the running maximum - SHIFT; m is raised (and the row's O
    // rescaled) only when a block's maximum exceeds it by more than RESCALE base-2 units, so P stays below
    // 2^(SHIFT + RESCALE). In FP16 that uses the range up to 2^15: weights keep their 11 bits down to 2^-25 of the largest
    // and vanish below 2^-36, so that a long context behind a key far ahead of it is not lost (with m = the maximum
    // itself, below 2^-25: 32767 keys 17.4 natural units behind one summed to nothing). BF16 has FP32's range.
    static constexpr float SHIFT = std::is_same<T, __half>::value ? 11.0f : 0.0f;
    static constexpr float RESCALE = std::is_same<T, __half>::value ? 4.0f : 8.0f;
    static constexpr int SMEM_BYTES = 1024 + BAR_OFF + NUM_BARS * 8 + 16;
    static constexpr int NUM_THREADS = 64 + NT * 128;
    // Warps: the softmax warps of the tiles (warp w reads the Tensor Memory lanes of quarter w mod 4),
    // then the MMA issuer and the producer
    static constexpr int MMA_WARP = 4 * NT, PRODUCER_WARP = 4 * NT + 1;
    static constexpr int CTAS_PER_SM = NT == 1 ? 2 : 1;
    // TMEM: NT = 1: two score buffers of 64 columns, O; NT = 2: S_A S_B O_A O_B. P (16-bit pairs)
    // over the first half of its scores.
    static constexpr int S_COL = 0, O_COL = 2 * BKV;
    static constexpr int TMEM_COLS = NT == 1 ? 256 : 512;
    static_assert(O_COL + NT * D <= TMEM_COLS, "Tensor Memory columns");
    static_assert(SMEM_BYTES + 1024 <= (NT == 1 ? 116736 : 233472), "shared memory of an SM");
    static constexpr uint32_t TYPE_BITS = std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
    // FP32 accumulation, M = 128, A K-major; S: N = BKV, B (keys) K-major; PV: N = D, B (values)
    // MN-major
    static constexpr uint32_t ID_S = (1u << 4) | TYPE_BITS | (static_cast<uint32_t>(BKV >> 3) << 17) | (128u >> 4 << 24);
    static constexpr uint32_t ID_PV = (1u << 4) | TYPE_BITS | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (128u >> 4 << 24);
};

// NT = 2: with fewer than kPagedCoarse blocks per CTA, items are cut at multiples of kPagedQuantum
// blocks only: a part costs about as much (128 KB of FP32 written and read again) as the blocks.
constexpr int kPagedCoarse = 8, kPagedLog2Quantum = 2, kPagedQuantum = 1 << kPagedLog2Quantum;

// 2^(s - m) is off by as much for all keys of a row as m is rounded, which the sums take out again: as long as that is
// little. From this |m| on (half a step of 2^-12; scores of 2840) the raw scores are made relative to the one that m comes
// from before they are scaled, so that what m rounds to plays no part (a score of 2^26 lies up to 4 off its rounded m,
// which FP16's P does not hold). Costs ordinary scores a comparison and a vote more per block: prompts 148.3 -> 149.9 us,
// drafts 78.5 -> 79.9.
constexpr float kPagedLarge = 4096.0f;

// ---- work units --------------------------------------------------------------------------------
//
// (compiled for the host too, so that the ranges can be checked without a GPU)

// sum over i < n of floor((a i + b) / 2^k), a > 0, b >= 0. Twos that a has are taken out of both sides. An odd a meets
// each remainder mod P = 2^k once in P steps, so these sum to (a - 1)(P - 1) / 2 + b, the next P to a P more, and
// so on; the steps after the last whole P (fewer than 2^k, with k at most 9; few or none for a power of two) are added up.
__host__ __device__ __noinline__ int64_t sum_of_shares(int64_t n, int k, int a, int64_t b)
{
#pragma unroll 1
    for (; k > 0 && a % 2 == 0; --k) {
        a /= 2;
        b >>= 1;
    }
    const int64_t times = n >> k;
    const int rest = static_cast<int>(n - (times << k)), low = static_cast<int>(b & ((1 << k) - 1));
    const int64_t first = static_cast<int64_t>(a - 1) * ((1 << k) - 1) / 2 + b;
    int64_t sum = times * first + times * (times - 1) / 2 * (static_cast<int64_t>(a) << k) + rest * (times * a + (b >> k));
#pragma unroll 1
    for (int i = 0; i < rest; ++i)
        sum += (a * i + low) >> k;
    return sum;
}

// The items of one sequence (or the prefix items, of all tokens together): tiles of `step` tokens
// for each key head. `edge`: keys that the token before the first would see, counted from the
// items' first key (token i sees the edge + i + 1 first of them); fixed >= 0: every tile has
// `fixed` blocks instead.
struct SeqItems {
    int q0, n, kv, tiles, fixed;
    int edge, step;
    bool bad;
    __host__ __device__ bool prefix() const { return fixed >= 0; }
};

// Sequences of a launch, the prefix counted as one; number s of them.
__host__ __device__ __forceinline__ int seq_count(const PagedParams &p)
{
    return p.keys == KEYS_PREFIX ? 1 : p.keys == KEYS_BOTH ? p.batch.num_seqs + 1 : p.batch.num_seqs;
}

template <class Cfg>
__host__ __device__ __noinline__ SeqItems seq_items(const PagedParams &p, int s)
{
    SeqItems q;
    if (p.keys == KEYS_PREFIX || (p.keys == KEYS_BOTH && s == 0)) {
        const int a = min(max(load_int(p.batch.q_start), 0), p.batch.num_tokens);
        const int b = min(max(load_int(p.batch.q_start + p.batch.num_seqs), a), p.batch.num_tokens);
        q.q0 = a;
        q.n = b - a;
        q.kv = 0;
        q.fixed = (p.batch.prefix_len + Cfg::BKV - 1) / Cfg::BKV;
        q.edge = 0;
        q.step = Cfg::NT * p.long_tokens;
        q.bad = false;
        q.tiles = (q.n + q.step - 1) / q.step;
        return q;
    }
    const SeqView v = load_seq(p.batch, p.keys == KEYS_BOTH ? s - 1 : s);
    q.q0 = v.q0;
    q.n = v.n;
    q.kv = v.kv;
    q.fixed = -1;
    q.edge = (p.keys == KEYS_ALL ? p.batch.prefix_len : 0) + v.kv - v.n;
    q.step = Cfg::NT * p.tile_tokens;
    q.bad = v.bad;
    const bool mine = p.seqs == SEQS_ALL || (v.n > p.long_tokens) == (p.seqs == SEQS_LONG);
    q.tiles = mine ? (v.n + q.step - 1) / q.step : 0;
    return q;
}

// Key blocks of the tokens [.., last] (at least one, so that rows that see nothing are written).
template <class Cfg>
__host__ __device__ __forceinline__ int blocks_upto(const SeqItems &q, int last)
{
    if (q.fixed >= 0)
        return q.fixed;
    return max(1, (q.edge + last + Cfg::BKV) / Cfg::BKV);
}

// Units of the tile whose last token is `last`: its blocks and, ahead of them, what beginning an
// item costs (ITEM_COST blocks' time), in steps of `quantum` (the last maybe fewer). A range that
// ends within the cost leaves the whole item to the next.
template <class Cfg>
__host__ __device__ __forceinline__ int units_upto(const SeqItems &q, int quantum, int last)
{
    return (blocks_upto<Cfg>(q, last) + Cfg::ITEM_COST + quantum - 1) / quantum;
}

// First block of an item's unit `u`.
template <class Cfg>
__host__ __device__ __forceinline__ int block_of(int u, int quantum, int blocks)
{
    return min(blocks, max(0, u * quantum - Cfg::ITEM_COST));
}

// Units of all tiles of one key head.
template <class Cfg>
__host__ __device__ inline int64_t units_of_head(const SeqItems &q, int quantum)
{
    const int step = q.step;
    if (q.tiles == 0)
        return 0;
    const int last = units_upto<Cfg>(q, quantum, q.n - 1);
    if (q.fixed >= 0 || q.tiles == 1)
        return static_cast<int64_t>(q.tiles) * last;
    // the tiles before the last: tile t sees the edge + (t + 1) step first keys, at least one block's
    const int whole = q.tiles - 1, keys = Cfg::BKV * quantum;
    const int ones = min(whole, max(0, (Cfg::BKV - q.edge) / step));
    int64_t sum = last + static_cast<int64_t>(ones) * ((1 + Cfg::ITEM_COST + quantum - 1) / quantum);
    if (whole > ones) {
        const int64_t b = static_cast<int64_t>(q.edge) + static_cast<int64_t>(ones + 1) * step + Cfg::ITEM_COST * Cfg::BKV + keys - 1;
        sum += sum_of_shares(whole - ones, (Cfg::BKV == 64 ? 6 : 7) + (quantum == 1 ? 0 : kPagedLog2Quantum), step, b);
    }
    return sum;
}

// A CTA's walk over the units of its range.
struct Walk {
    int s;            // see seq_items()
    SeqItems q;
    int head, tile, unit, quantum;
    int64_t left;     // units left in the range
};

// One stretch of an item: key blocks [b0, b1) of `blocks`.
struct Segment {
    bool prefix;               // keys of the prefix
    int s, head, tok0, toks;   // sequence; tokens [tok0, tok0 + toks) of the flat dimension
    int tile_tokens;           // per tile
    int q0, kv, edge;          // see SeqItems
    int b0, b1, blocks;
    int units;                 // of the item
    int64_t ahead;             // from the item's first unit to the end of the CTA's range

    // Tokens of a tile: the first (of the item's) and how many. The only tile of an item is the
    // last one, so that the barriers it completes are always the same.
    template <int NT>
    __host__ __device__ int tile_first(int tile) const { return NT == 1 || toks <= tile_tokens ? 0 : tile * tile_tokens; }
    template <int NT>
    __host__ __device__ int tile_toks(int tile) const
    {
        return NT == 2 && tile == 0 && toks <= tile_tokens ? 0 : min(tile_tokens, toks - tile_first<NT>(tile));
    }
    // Its blocks: the first tile of two may see fewer keys than the second.
    template <int NT, int BKV>
    __host__ __device__ int tile_blocks(int tile) const
    {
        if (NT == 1 || tile == 1)
            return blocks;
        if (toks <= tile_tokens)
            return 0;
        return prefix ? blocks : max(1, (edge + (tok0 + tile_tokens - 1 - q0) + BKV) / BKV);
    }
};

template <class Cfg>
__host__ __device__ __forceinline__ bool next_segment(const PagedParams &p, Walk &w, Segment &g)
{
    do {
        if (w.left <= 0)
            return false;
        while (w.tile >= w.q.tiles) {   // on to the next head or the next sequence with items (units are left)
            if (w.q.tiles > 0 && w.head + 1 < p.kv_heads) {
                ++w.head;
            } else {
                w.head = 0;
                if (++w.s >= seq_count(p))
                    return false;
                w.q = seq_items<Cfg>(p, w.s);
            }
            w.tile = 0;
        }
        const int first = w.tile * w.q.step, toks = min(w.q.step, w.q.n - first);
        g.prefix = w.q.prefix();
        g.s = p.keys == KEYS_BOTH ? w.s - 1 : w.s;
        g.tile_tokens = w.q.step / Cfg::NT;
        g.head = w.head;
        g.tok0 = w.q.q0 + first;
        g.toks = toks;
        g.q0 = w.q.q0;
        g.kv = w.q.kv;
        g.edge = w.q.edge;
        g.blocks = blocks_upto<Cfg>(w.q, first + toks - 1);
        g.units = (g.blocks + Cfg::ITEM_COST + w.quantum - 1) / w.quantum;
        const int u1 = static_cast<int>(min(static_cast<int64_t>(g.units), w.unit + w.left));
        g.b0 = block_of<Cfg>(w.unit, w.quantum, g.blocks);
        g.b1 = block_of<Cfg>(u1, w.quantum, g.blocks);
        g.ahead = w.left + w.unit;
        w.left -= u1 - w.unit;
        if (u1 == g.units) {
            ++w.tile;
            w.unit = 0;
        } else {
            w.unit = u1;   // the range ends here
        }
    } while (g.b0 == g.b1);   // (units of the item's cost only)
    return true;
}

// The tile of `q` that holds unit `at` of a key head, found by `threads` threads together, `thread` of
// them this one: scan(value, ahead) returns the sum of value over all and sets ahead to that over the
// threads before this one. One thread calls found(tile, unit of the tile). A head's units pass 32 bits (2^31 of
// them: a prompt of 1.04 million tokens, 128 query heads to a key head), those of a tile do not.
template <class Cfg, class Scan, class Found>
__host__ __device__ __forceinline__ void locate_tile(const SeqItems &q, int quantum, int64_t at, int thread, int threads, Scan &&scan,
                                                     Found &&found)
{
    int64_t done = 0;
    for (int t0 = 0; t0 < q.tiles && done <= at; t0 += threads) {
        const int t = t0 + thread;
        const int units = t < q.tiles ? units_upto<Cfg>(q, quantum, min((t + 1) * q.step, q.n) - 1) : 0;
        int64_t first;
        const int64_t all = scan(static_cast<int64_t>(units), first);
        if (units > 0 && done + first <= at && at < done + first + units)
            found(t, static_cast<int>(at - done - first));
        done += all;
    }
}

// What the CTAs agree on: `total` units over `ctas` non-empty ranges.
struct Shares {
    int64_t total;
    int ctas;
    __host__ __device__ int64_t begin(int c) const { return total * c / ctas; }
    // the range that holds unit u
    __host__ __device__ int owner(int64_t u) const { return static_cast<int>(((u + 1) * ctas + total - 1) / total) - 1; }
};

// Position in the ring of query buffers (their number is the launch's).
struct QueryPos {
    int bufs, buf = 0;
    uint32_t parity = 0;
    __device__ explicit QueryPos(int n) : bufs(n) {}
    __device__ void step()
    {
        if (++buf == bufs) {
            buf = 0;
            parity ^= 1u;
        }
    }
};

// Ring position of the K/V tiles.
template <int N>
struct RingPos {
    int slot = 0;
    uint32_t parity = 0;
    __device__ void step()
    {
        if (++slot == N) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// ---- softmax warp ------------------------------------------------------------------------------

// Reads the columns addr .. addr + 32 N - 1 of this warp's TMEM lanes in chunks of 32 and hands
// each to fn(registers, chunk). Warp-collective. A loop, one load at a time: unrolled, with the
// next load in flight, the softmax waits for instructions instead (prompts 151.2 against 160.5 us,
// drafts 80.6 against 83.2).
template <int N, class Fn>
__device__ __forceinline__ void tmem_chunks(uint32_t addr, uint32_t (&v)[32], Fn &&fn)
{
#pragma unroll 1
    for (int c = 0; c < N; ++c) {
        tmem_ld_32x32b_x32(addr + 32u * c, v);
        tmem_ld_wait_regs(v);
        fn(v, c);
    }
}

// Subtracts x from 32 N columns of this warp's lanes.
template <int N>
__device__ __forceinline__ void subtract_scores(uint32_t addr, float x)
{
    uint32_t v[32];
#pragma unroll 1
    for (int c = 0; c < N; ++c) {
        tmem_ld_32x32b_x32(addr + 32u * c, v);
        tmem_ld_wait_regs(v);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] = __float_as_uint(__uint_as_float(v[e]) - x);
        tmem_st_32x32b_x32(addr + 32u * c, v);
    }
    tmem_st_wait();
}

// Every lane of the warp has 128 bytes (8 pieces) for its address `row` (16-byte aligned; nullptr:
// none): they go through the warp's 4 KB at `stage`, so that 8 lanes write one row's 128 bytes
// (piece k of row r at k ^ (r mod 8): no bank conflicts either way). Stored a row per lane, each
// store instruction touches 32 lines, 16 bytes in each.
__device__ __forceinline__ void store_rows(uint32_t stage, int lane, const uint4 (&piece)[8], char *row)
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        st_shared_v4(stage + static_cast<uint32_t>(lane) * 128u + static_cast<uint32_t>(k ^ (lane & 7)) * 16u, piece[k]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + lane / 8, k = lane & 7;
        const float4 v = ld_shared_f4(stage + static_cast<uint32_t>(r) * 128u + static_cast<uint32_t>(k ^ (r & 7)) * 16u);
        char *dst = reinterpret_cast<char *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r));
        if (dst)
            *reinterpret_cast<float4 *>(dst + 16 * k) = v;
    }
    __syncwarp();
}

struct PagedBars {
    uint32_t q_full0, q_empty0, drain, full0, empty0, s_full, pv_done, p_half0, p_full0;
};

// Keys of the prefix that a token sees: normally all; one that stands inside it sees less. Of a
// warp whose tokens do not decrease (not inlined: the items of a batch's own keys never call it,
// and the instruction cache is what short items wait for). All lanes call it.
__device__ __noinline__ int prefix_seen(const BatchView &b, int token, bool on)
{
    int s = find_seq<32>(b.q_start, b.num_seqs, __shfl_sync(0xffffffffu, token, 0), threadIdx.x & 31);
    if (!on)
        return 0;
    while (s + 1 < b.num_seqs && __ldg(b.q_start + s + 1) <= token)
        ++s;
    const SeqView v = load_seq(b, s);
    return min(b.prefix_len, max(0, b.prefix_len + v.kv - v.n + (token - v.q0) + 1));
}

// (m, l) of a part as it is kept. Of no weight is l = 0; m is NaN then if the row sees a key of the part all the same (scores of
// -inf only): its O counts, 0 unless a value is not finite, and the row is 0/0 if all its parts are such. With any other
// m the part has no key for the row: its O may not be written, and a row of such parts only is 0.
__device__ __forceinline__ float2 part_ml(float m, float l, bool sees)
{
    return make_float2(l == 0.0f && sees ? NAN : m, l);
}

__device__ __forceinline__ bool no_key(float2 ml) { return ml.y == 0.0f && ml.x == ml.x; }

// A key that some rows of an item see and others do not gets P = 0 for those, and 0 times a value
// that is infinite or NaN is NaN. So a warp that finds such an O in a row that does not see all keys of
// its stretch goes through the CTA's stretches once more when it is done, and computes the rows that such
// a value has spoilt anew, over the keys that they see and no others: kRepairRows rows at a time, a lane
// holding D / 32 dimensions of all of them, so that a key and its value are fetched once for all;
// kRepairKeys keys at a time, those after them in flight. A NaN in the last key of a prompt of 4096 tokens behind 32
// heads (128 rows each over all keys): 6.9 ms, 71 with a row at a time (0.15 without the NaN); in every last key of a
// mixed step 9.7, 101. Bound by latency, 193 instructions a key and group of rows at 4 clocks each, one warp to a
// scheduler. Hardly ever anything, and not inlined; what it costs
// otherwise is the look at O, instructions to fetch at the end of each such item (drafts 71.7 -> 76.6 us, shared
// step 52.4 -> 53.0, prompts the same).
constexpr int kRepairRows = 8, kRepairKeys = 4;

// Sums of x[0 .. 7] over the warp: lane i gets that of x[i / 4].
__device__ __forceinline__ float sum_rows(float (&x)[8], int lane)
{
#pragma unroll
    for (int n = 4; n > 0; n /= 2) {
        const bool upper = lane & (4 * n);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? x[i] : x[i + n];
            x[i] = (upper ? x[i + n] : x[i]) + __shfl_xor_sync(0xffffffffu, send, 4 * n);
        }
    }
    x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

template <class Cfg>
__device__ __noinline__ void repair_stretches(const PagedParams &p, const Walk &start, int tile, int quarter, int lane)
{
    using T = typename Cfg::Type;
    constexpr int D = Cfg::D, BKV = Cfg::BKV, V = D / 32;   // a lane's dims: lane * V ..
    constexpr int R = kRepairRows, KEYS = kRepairKeys;
    constexpr uint32_t ALL = 0xffffffffu;
    struct Vec {
        uint32_t w[V / 2];
    };
    auto fetch = [&](const void *base, int64_t at) -> Vec {   // this lane's dims of the vector there; at < 0: zeros
        Vec x = {};
        if (at >= 0) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const T *>(base) + at + lane * V);
#pragma unroll
            for (int e = 0; e < V / 2; ++e)
                x.w[e] = src[e];
        }
        return x;
    };
    auto unpack = [](const Vec &x, float(&f)[V]) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 y = unpack2<T>(x.w[e / 2]);
            f[e] = y.x;
            f[e + 1] = y.y;
        }
    };
    Walk walk = start;
    Segment g;
    while (next_segment<Cfg>(p, walk, g)) {
        const int first = g.tile_first<Cfg::NT>(tile), toks = g.tile_toks<Cfg::NT>(tile);
        const int alive = g.prefix ? p.batch.prefix_len : max(0, g.edge + (g.tok0 + g.toks - g.q0));
        const int begin = g.b0 * BKV, end = min(min(g.b1, g.tile_blocks<Cfg::NT, BKV>(tile)) * BKV, alive);
        const int key_base = g.prefix || p.keys == KEYS_ALL ? 0 : p.batch.prefix_len;
        const bool starts = g.b0 == 0, whole = starts && g.b1 == g.blocks;
        const bool final_row = whole && p.keys == KEYS_ALL;
        // element of the cache where the vector of key j is; -1: of a bad page (which counts as zeros), or past `last`
        auto place = [&](int j, int last) -> int64_t {
            if (j >= last)
                return -1;
            const int key = key_base + j, lp = key >> p.batch.page_shift;
            const int page = lp < p.n_prefix_pages ? __ldg(p.prefix_pages + lp)
                                                   : __ldg(p.batch.table + g.s * p.batch.table_stride + (lp - p.n_prefix_pages));
            return page < 0 || page >= p.batch.num_pages
                       ? -1
                       : page * p.page_stride + g.head * p.head_stride + (key & ((1 << p.batch.page_shift) - 1)) * p.row_stride;
        };
        // this lane's row, and where its O and (m, l) are
        const int r = quarter * 32 + lane, token = g.tok0 + first + r / p.group, head = g.head * p.group + r % p.group;
        const bool on = r / p.group < toks;
        int seen;
        if (g.prefix)
            seen = prefix_seen(p.batch, token, on);
        else
            seen = on ? max(0, g.edge + (token - g.q0) + 1) : 0;
        const uint32_t some = __ballot_sync(ALL, on && seen > begin && seen < end);   // not all of the stretch, and not none
        if (some == 0)
            continue;
        const int64_t row =
            whole ? static_cast<int64_t>(token) * (p.kv_heads * p.group) + head
                  : (static_cast<int64_t>(2 * blockIdx.x + (starts ? 1 : 0)) * p.parts.tiles + (first > 0 ? 1 : 0)) * p.parts.rows + r;
        const int64_t at_o = final_row ? token * p.out_token + head * p.out_head : row * D;   // elements
        float *const part_o = whole ? p.row_o[g.prefix] : p.parts.o;
        // the last key of the stretch whose value is not finite in each dim, among those that not all rows see:
        // a row that sees it is as it should be
        int bad[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            bad[e] = -1;
        const int hidden = __reduce_min_sync(ALL, some >> lane & 1u ? seen : INT32_MAX);
        for (int j0 = hidden; j0 < end; j0 += 32) {
            const int64_t mine = place(j0 + lane, end);
#pragma unroll 4
            for (int i = 0; i < 32; ++i) {
                float v[V];
                unpack(fetch(p.v, __shfl_sync(ALL, mine, i)), v);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    bad[e] = fabsf(v[e]) < INFINITY ? bad[e] : j0 + i;
            }
        }
        uint32_t rows = 0;
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {
            const int64_t at = __shfl_sync(ALL, at_o, i);
            const int n = __shfl_sync(ALL, seen, i);
            float x[V] = {};
            if (some >> i & 1u) {
                if (final_row) {
                    unpack(fetch(p.out, at), x);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        x[e] = part_o[at + lane * V + e];
                }
            }
            bool spoilt = false;
#pragma unroll
            for (int e = 0; e < V; ++e)
                spoilt = spoilt || (bad[e] >= n && !(fabsf(x[e]) < INFINITY));
            rows |= __any_sync(ALL, spoilt) && (some >> i & 1u) ? 1u << i : 0u;
        }
        while (rows) {
            // the next R rows (or what there is: then the last one again, not written)
            int lanes[R], count = 0, mine = 0;
            float q[R][V], acc[R][V];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (rows) {
                    lanes[i] = __ffs(static_cast<int>(rows)) - 1;
                    rows &= rows - 1;
                    ++count;
                } else {
                    lanes[i] = lanes[i > 0 ? i - 1 : 0];
                }
                mine = lane / 4 == i ? lanes[i] : mine;
                const int from = quarter * 32 + lanes[i];
                unpack(fetch(p.q, (g.tok0 + first + from / p.group) * p.q_token + (g.head * p.group + from % p.group) * p.q_head), q[i]);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    acc[i][e] = 0.0f;
            }
            // of row lane / 4: keys it sees, running maximum (raised beyond 2^8, as in the softmax) and sum
            const int sees = __shfl_sync(ALL, seen, mine), last = __reduce_max_sync(ALL, sees);
            float m = -INFINITY, l = 0.0f;
            for (int j0 = begin; j0 < last; j0 += 32) {
                const int64_t at = place(j0 + lane, last);
                Vec k[KEYS], v[KEYS];
#pragma unroll
                for (int u = 0; u < KEYS; ++u) {
                    k[u] = fetch(p.k, __shfl_sync(ALL, at, u));
                    v[u] = fetch(p.v, __shfl_sync(ALL, at, u));
                }
#pragma unroll 1
                for (int i0 = 0; i0 < 32 && j0 + i0 < last; i0 += KEYS) {
                    float score[KEYS], top = -INFINITY;
                    Vec now[KEYS];   // the values of these keys
#pragma unroll
                    for (int u = 0; u < KEYS; ++u) {
                        float kf[V], x[R];
                        unpack(k[u], kf);
                        now[u] = v[u];
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            x[i] = q[i][0] * kf[0];
#pragma unroll
                            for (int e = 1; e < V; ++e)
                                x[i] = fmaf(q[i][e], kf[e], x[i]);
                        }
                        score[u] = sum_rows(x, lane) * p.scale_log2;
                        top = j0 + i0 + u < sees ? fmaxf(top, score[u]) : top;   // (a NaN score leaves it alone)
                        // the same of the next KEYS keys (past this step's 32: fetched above, when it comes)
                        const int64_t next = __shfl_sync(ALL, at, (i0 + KEYS + u) & 31);
                        if (i0 + KEYS < 32) {
                            k[u] = fetch(p.k, next);
                            v[u] = fetch(p.v, next);
                        }
                    }
                    const bool raise = top > m + 8.0f;
                    if (__any_sync(ALL, raise)) {
                        const float keep = raise ? exp2f(m - top) : 1.0f;
                        m = raise ? top : m;
                        l *= keep;
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float x = __shfl_sync(ALL, keep, 4 * i);
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                acc[i][e] *= x;
                        }
                    }
                    const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int u = 0; u < KEYS; ++u) {
                        const bool on_key = j0 + i0 + u < sees;
                        const float w = on_key ? exp2f(score[u] - from) : -1.0f;   // -1: not seen
                        l += on_key ? w : 0.0f;
                        float vf[V];
                        unpack(now[u], vf);
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float x = __shfl_sync(ALL, w, 4 * i);
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                acc[i][e] = x == -1.0f ? acc[i][e] : fmaf(x, vf[e], acc[i][e]);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t at = __shfl_sync(ALL, at_o, lanes[i]), at_ml = __shfl_sync(ALL, row, lanes[i]);
                const float mi = __shfl_sync(ALL, m, 4 * i), li = __shfl_sync(ALL, l, 4 * i), inv = 1.0f / li;
                if (i >= count)
                    continue;
                if (final_row) {
                    T *out = static_cast<T *>(p.out) + at + lane * V;
#pragma unroll
                    for (int e = 0; e < V; e += 2)
                        *reinterpret_cast<uint32_t *>(out + e) = pack2<T>(acc[i][e] * inv, acc[i][e + 1] * inv);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        part_o[at + lane * V + e] = acc[i][e];
                    if (lane == 0)
                        (whole ? p.row_ml[g.prefix] : p.parts.ml)[at_ml] = part_ml(mi, li, true);
                }
            }
        }
    }
}

template <class Cfg>
__device__ __forceinline__ void paged_softmax_warp(const PagedParams &p, const PagedBars &bar, const WaitCtl &wc, uint32_t tmem,
                                                   uint32_t ring, uint32_t stage, volatile int *spoilt, volatile float *ref, const Walk &start,
                                                   const Shares &shares, int tile, int warp, int lane)
{
    using T = typename Cfg::Type;
    constexpr int D = Cfg::D, BKV = Cfg::BKV, CH = BKV / 32;
    // The last tile's scores and products complete the ring's barriers (its K or V tile is free
    // then, too); the first of two tiles has barriers of its own.
    const bool last_tile = tile == Cfg::NT - 1;
    const int quarter = warp & 3;
    if (quarter >= p.busy_warps)
        return;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_addr = tmem + lane_base + static_cast<uint32_t>(Cfg::O_COL + tile * D);
    const int row_tok = r / p.group, row_head = r - row_tok * p.group;   // token of the tile, head of the group
    const float sl2 = p.scale_log2;   // not 0 (the host sees to it): a masked score times it is -inf
    const uint32_t hidden = __float_as_uint(sl2 >= 0.0f ? -INFINITY : INFINITY);
    const uint32_t p_half = bar.p_half0 + 8u * tile;
    RingPos<Cfg::STAGES> ring_k;   // this block's K tile (its V tile is the next position)
    uint32_t count = 0;            // blocks this tile has worked on
    uint32_t va[32], vb[32];
    Walk walk = start;
    Segment g, next;
    bool more = next_segment<Cfg>(p, walk, next);
    while (more) {
        g = next;
        // ---- rows and masks of the stretch
        const int first = g.tile_first<Cfg::NT>(tile), toks = g.tile_toks<Cfg::NT>(tile);
        const bool row_ok = row_tok < toks;
        const int token = g.tok0 + first + row_tok;
        int seen = INT32_MAX;   // keys, from the item's first, that the row sees (idle rows: as if all)
        if (g.prefix) {
            const int n = prefix_seen(p.batch, token, row_ok);
            seen = row_ok ? n : seen;
        } else if (row_ok) {
            seen = max(0, g.edge + (token - g.q0) + 1);
        }
        const bool active = __any_sync(0xffffffffu, row_ok);
        // keys that any row of the item sees: rows of V past them are zeroed
        const int alive = g.prefix ? p.batch.prefix_len : max(0, g.edge + (g.tok0 + g.toks - g.q0));
        const int mine = g.tile_blocks<Cfg::NT, BKV>(tile);
        float m = -INFINITY, l = 0.0f;
        bool any_block = false;
        RingPos<Cfg::STAGES> prev_v = ring_k;
        for (int b = g.b0; b < g.b1; ++b) {
            RingPos<Cfg::STAGES> ring_v = ring_k;
            ring_v.step();
            if (b >= mine) {   // the other tile's blocks only
                ring_k = ring_v;
                ring_k.step();
                continue;
            }
            if (!(last_tile ? wait_warp(bar.empty0 + 8u * ring_k.slot, ring_k.parity, wc, ERR_EPILOGUE_ACCUMULATOR, lane)
                            : wait_warp(bar.s_full, count & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane)))
                return;
            tc_fence_after_sync();
            const int k0 = b * BKV;
            if (k0 + BKV > alive) {
                // rows of V that no row sees: zero them once the tile has landed
                if (!wait_warp(bar.full0 + 8u * ring_v.slot, ring_v.parity, wc, ERR_EPILOGUE_ACCUMULATOR, lane))
                    return;
                const uint32_t v_tile = ring + static_cast<uint32_t>(ring_v.slot) * Cfg::KV_TILE;
                const int from = max(0, alive - k0);
                for (int i = from * 8 + r; i < BKV * 8; i += 32 * p.busy_warps)
#pragma unroll
                    for (int a = 0; a < Cfg::ATOMS; ++a)
                        st_shared_v4(v_tile + static_cast<uint32_t>(a) * Cfg::KV_ATOM + static_cast<uint32_t>(i) * 16u,
                                     make_uint4(0, 0, 0, 0));
                fence_proxy_async_shared();
            }
            const uint32_t s_addr =
                tmem + lane_base + static_cast<uint32_t>(Cfg::S_COL + (Cfg::NT == 1 ? static_cast<int>(count & 1u) : tile) * BKV);
            if (active) {
                // Masked scores are overwritten in TMEM first, 32 keys at a time, only where a key is
                // masked for some row of the warp: the code below, which every block runs, stays the
                // only copy (a second, masked one was fetched anew at every item's end: 2.8 us a block
                // against 0.95).
                if (!__all_sync(0xffffffffu, k0 + BKV <= seen)) {
#pragma unroll 1
                    for (int c = 0; c < CH; ++c) {
                        const int lim = seen - k0 - 32 * c;   // keys of these 32 that the row sees
                        if (__all_sync(0xffffffffu, lim >= 32))
                            continue;
                        if (__any_sync(0xffffffffu, row_ok && lim > 0)) {
                            tmem_ld_32x32b_x32(s_addr + 32u * c, va);
                            tmem_ld_wait_regs(va);
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            va[e] = e < lim ? va[e] : hidden;
                        tmem_st_32x32b_x32(s_addr + 32u * c, va);
                    }
                    tmem_st_wait();
                }
                // the extreme of the raw scores in four independent chains, scaled once
                float r0 = sl2 >= 0.0f ? -INFINITY : INFINITY, r1 = r0, r2 = r0, r3 = r0;
                tmem_chunks<CH>(s_addr, va, [&](const uint32_t(&x)[32], int) {
                    if (sl2 >= 0.0f) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            r0 = fmax3(r0, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                            r1 = fmax3(r1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                            r2 = fmax3(r2, __uint_as_float(x[e + 4]), __uint_as_float(x[e + 5]));
                            r3 = fmax3(r3, __uint_as_float(x[e + 6]), __uint_as_float(x[e + 7]));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            r0 = fmin3(r0, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                            r1 = fmin3(r1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                            r2 = fmin3(r2, __uint_as_float(x[e + 4]), __uint_as_float(x[e + 5]));
                            r3 = fmin3(r3, __uint_as_float(x[e + 6]), __uint_as_float(x[e + 7]));
                        }
                    }
                });
                const float rb = sl2 >= 0.0f ? fmax3(fmaxf(r0, r1), r2, r3) : fmin3(fminf(r0, r1), r2, r3);
                const float mb = rb * sl2 - Cfg::SHIFT;
                const bool raise = mb > m + Cfg::RESCALE || m == -INFINITY;
                float m_new = raise ? mb : m;
                float m_use = m_new == -INFINITY ? 0.0f : m_new;
                float alpha = raise && row_ok ? ex2_approx(m - m_use) : 1.0f;   // 0 on the first block
                const bool large = row_ok && fabsf(m_use) > kPagedLarge;
                if (__any_sync(0xffffffffu, large || (any_block && alpha != 1.0f))) {
                    if (__builtin_expect(__any_sync(0xffffffffu, large), 0)) {
                        if (large) {
                            bool up = raise;
                            if (m != -INFINITY && fabsf(m) > kPagedLarge) {   // (then *ref is what m comes from)
                                up = (rb - *ref) * sl2 > Cfg::RESCALE;
                                m_new = up ? mb : m;
                                alpha = up ? ex2_approx((*ref - rb) * sl2) : 1.0f;
                            }
                            if (up)
                                *ref = rb;
                            m_use = -Cfg::SHIFT;
                        }
                        subtract_scores<CH>(s_addr, large ? *ref : 0.0f);
                    }
                    if (any_block) {
                        // O holds the blocks before: once their product is complete, rescale the rows
                        if (!(last_tile ? wait_warp(bar.empty0 + 8u * prev_v.slot, prev_v.parity, wc, ERR_EPILOGUE_ACCUMULATOR, lane)
                                        : wait_warp(bar.pv_done, (count - 1u) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane)))
                            return;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            tmem_ld_32x32b_x32(o_addr + 32u * c, va);
                            tmem_ld_wait_regs(va);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                va[e] = __float_as_uint(__uint_as_float(va[e]) * alpha);
                            tmem_st_32x32b_x32(o_addr + 32u * c, va);
                        }
                        tmem_st_wait();
                    }
                }
                uint64_t sum2[4] = {f32x2_pack(0.0f, 0.0f), f32x2_pack(0.0f, 0.0f), f32x2_pack(0.0f, 0.0f),
                                    f32x2_pack(0.0f, 0.0f)};
                const uint64_t scale2 = f32x2_pack(sl2, sl2), neg_m2 = f32x2_pack(-m_use, -m_use);
                tmem_chunks<CH>(s_addr, va, [&](const uint32_t(&x)[32], int c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float t0, t1;
                        f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), scale2, neg_m2),
                                     t0, t1);
                        const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                        sum2[i & 3] = f32x2_add(sum2[i & 3], f32x2_pack(p0, p1));
                        pk[i] = pack2<T>(p0, p1);
                    }
                    tmem_st_32x32b_x16(s_addr + 16u * static_cast<uint32_t>(c), pk);   // over scores already read
                    if (Cfg::NT == 2 && c == CH / 2 - 1) {
                        // the first half of the keys: their product can start
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(p_half);
                    }
                });
                float s0, s1;
                f32x2_unpack(f32x2_add(f32x2_add(sum2[0], sum2[1]), f32x2_add(sum2[2], sum2[3])), s0, s1);
                l = l * alpha + (s0 + s1);
                m = m_new;
                tmem_st_wait();
            } else if (Cfg::NT == 2) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_half);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(Cfg::NT == 1 ? bar.p_half0 + 8u * (count & 1u) : bar.p_full0 + 8u * tile);
            any_block = true;
            ++count;
            prev_v = ring_v;
            ring_k = ring_v;
            ring_k.step();
        }
        more = next_segment<Cfg>(p, walk, next);   // (while the last product runs)
        // ---- the stretch's result
        const bool starts = g.b0 == 0, ends = g.b1 == g.blocks;
        const bool whole = starts && ends;
        if (starts && tile == 0 && quarter == 0 && (!ends || p.keys != KEYS_ALL)) {
            int parts = 1;
            if (!ends)   // (its last range holds its last unit)
                parts = shares.owner(shares.begin(blockIdx.x + 1) - g.ahead + g.units - 1) - static_cast<int>(blockIdx.x) + 1;
            if (p.keys == KEYS_ALL) {
                if (lane == 0)
                    p.cuts[blockIdx.x] = make_int4(g.tok0, g.toks, g.head, parts);
            } else {
                for (int t = lane; t < g.toks; t += 32)
                    p.info[g.prefix][static_cast<int64_t>(g.tok0 + t) * p.kv_heads + g.head] =
                        make_int4(static_cast<int>(blockIdx.x), parts, g.tok0, p.launch);
            }
        }
        if (!active)
            continue;
        if (any_block) {
            if (!(last_tile ? wait_warp(bar.empty0 + 8u * prev_v.slot, prev_v.parity, wc, ERR_EPILOGUE_ACCUMULATOR, lane)
                            : wait_warp(bar.pv_done, (count - 1u) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane)))
                return;
            tc_fence_after_sync();
        }
        const int head = g.head * p.group + row_head;
        // rows that do not see all keys of the stretch: is their O finite (that of NaN scores is not meant to be)
        const bool part_seen = row_ok && l == l && seen < min(min(g.b1, mine) * BKV, alive);
        if (__builtin_expect(__any_sync(0xffffffffu, part_seen), 0)) {
            float top0 = 0.0f, top1 = 0.0f;   // largest magnitudes, NaN if there is one
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                tmem_ld_32x32b_x32(o_addr + static_cast<uint32_t>(c), va);
                tmem_ld_wait_regs(va);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    top0 = fmax3_abs_nan(top0, __uint_as_float(va[e]), __uint_as_float(va[e + 1]));
                    top1 = fmax3_abs_nan(top1, __uint_as_float(va[e + 2]), __uint_as_float(va[e + 3]));
                }
            }
            if (__builtin_expect(part_seen && !(top0 < INFINITY && top1 < INFINITY), 0))
                spoilt[warp] = 1;
        }
        if (whole && p.keys == KEYS_ALL) {
            const float inv = 1.0f / l;
            T *dst = static_cast<T *>(p.out) + token * p.out_token + head * p.out_head;
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                tmem_ld_32x32b_x32(o_addr + static_cast<uint32_t>(c), va);
                tmem_ld_32x32b_x32(o_addr + static_cast<uint32_t>(c) + 32u, vb);
                tmem_ld_wait_regs(va);
                tmem_ld_wait_regs(vb);
                uint4 piece[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int k = 8 * (i & 3) + 2 * e;
                        const float a = __uint_as_float(i < 4 ? va[k] : vb[k]), bb = __uint_as_float(i < 4 ? va[k + 1] : vb[k + 1]);
                        w[e] = seen == 0 ? 0u : pack2<T>(a * inv, bb * inv);
                    }
                    piece[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (Cfg::NT == 2) {
                    store_rows(stage, lane, piece, row_ok ? reinterpret_cast<char *>(dst + c) : nullptr);
                } else if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(dst + c + 8 * i) = piece[i];
                }
            }
            if (row_ok && p.lse)
                p.lse[token * p.lse_token + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            continue;
        }
        float *dst;
        float2 *ml;
        if (whole) {
            const int64_t row = static_cast<int64_t>(token) * (p.kv_heads * p.group) + head;
            dst = p.row_o[g.prefix] + row * D;
            ml = p.row_ml[g.prefix] + row;
        } else {
            const int64_t row =
                (static_cast<int64_t>(2 * blockIdx.x + (starts ? 1 : 0)) * p.parts.tiles + (first > 0 ? 1 : 0)) * p.parts.rows + r;
            dst = p.parts.o + row * D;
            ml = p.parts.ml + row;
        }
        if (any_block) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                tmem_ld_32x32b_x32(o_addr + static_cast<uint32_t>(c), va);
                tmem_ld_wait_regs(va);
                uint4 piece[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    piece[i] = make_uint4(va[4 * i], va[4 * i + 1], va[4 * i + 2], va[4 * i + 3]);
                if (Cfg::NT == 2) {
                    store_rows(stage, lane, piece, row_ok ? reinterpret_cast<char *>(dst + c) : nullptr);
                } else if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(dst + c + 4 * i) = piece[i];
                }
            }
        }
        if (row_ok)
            *ml = part_ml(m, l, seen > g.b0 * BKV);
    }
    __syncwarp();
    if (__builtin_expect(spoilt[warp], 0))
        repair_stretches<Cfg>(p, start, tile, quarter, lane);
}

// ---- kernel ------------------------------------------------------------------------------------

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NUM_THREADS, Cfg::CTAS_PER_SM)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_qp,
                           const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                           const __grid_constant__ PagedParams p)
{
    constexpr int NT = Cfg::NT, ATOMS = Cfg::ATOMS, BKV = Cfg::BKV, STAGES = Cfg::STAGES;
    constexpr int WARPS = Cfg::NUM_THREADS / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t warp_sum[WARPS];
    __shared__ Walk start;
    __shared__ int64_t start_at;   // unit of the key head with which the range begins
    __shared__ float refs[128 * NT];   // of each row, the raw score that a large m comes from
    __shared__ int spoilt[4 * NT];   // of each softmax warp, see repair_stretches
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sp = smem_raw + (base - raw);
    const uint32_t sQ = base + Cfg::Q_OFF, ring = base + Cfg::RING_OFF;
    PagedBars bar;
    bar.q_full0 = base + Cfg::BAR_OFF;
    bar.q_empty0 = bar.q_full0 + 8u * Cfg::Q_BUFS;
    bar.drain = bar.q_empty0 + 8u * Cfg::Q_BUFS;
    bar.full0 = bar.drain + 8u;
    bar.empty0 = bar.full0 + 8u * STAGES;
    bar.s_full = bar.empty0 + 8u * STAGES;
    bar.pv_done = bar.s_full + 8u;
    bar.p_half0 = bar.pv_done + 8u;
    bar.p_full0 = bar.p_half0 + 8u * NT;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sp + Cfg::BAR_OFF + Cfg::NUM_BARS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * Cfg::Q_BUFS; ++i)
            mbar_init(bar.q_full0 + 8u * i, 1);
        mbar_init(bar.drain, 1);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar.full0 + 8u * s, 1);
            mbar_init(bar.empty0 + 8u * s, 1);
        }
        mbar_init(bar.s_full, 1);
        mbar_init(bar.pv_done, 1);
        for (int t = 0; t < NT; ++t) {
            mbar_init(bar.p_half0 + 8u * t, static_cast<uint32_t>(p.busy_warps));   // the tile's softmax warps
            mbar_init(bar.p_full0 + 8u * t, static_cast<uint32_t>(p.busy_warps));
        }
        *abort_flag = 0;
        start.left = 0;
        for (int w = 0; w < 4 * NT; ++w)
            spoilt[w] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == Cfg::MMA_WARP) {
        tmem_alloc<1>(smem_u32(tmem_slot), Cfg::TMEM_COLS);
        tmem_relinquish<1>();
    }
    grid_dependency_wait();   // nothing above touched global memory

    // ---- this CTA's share of the units
    const int seqs = seq_count(p);
    // sum over the CTA's threads (block_sum, too), and over the threads before this one
    int64_t block_sum = 0;
    auto block_scan = [&](int64_t value, int64_t &ahead) -> int64_t {
        int64_t scan = value;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
            scan += lane >= o ? v : 0;
        }
        if (lane == 31)
            warp_sum[warp] = scan;
        __syncthreads();
        block_sum = 0;
        ahead = scan - value;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            ahead += w < warp ? warp_sum[w] : 0;
            block_sum += warp_sum[w];
        }
        __syncthreads();   // warp_sum may be written again
        return block_sum;
    };
    auto units_of = [&](int s, int quantum) -> int64_t {
        if (s >= seqs)
            return 0;
        const SeqItems q = seq_items<Cfg>(p, s);
        if (q.bad)
            atomicCAS(p.err, 0u, static_cast<uint32_t>(ERR_BATCH_INDEX));
        return p.kv_heads * units_of_head<Cfg>(q, quantum);
    };
    // units of the first chunk's sequence of this thread, those before it, and the sum over all
    int64_t own = 0, from = 0;
    auto add_up = [&](int quantum) -> int64_t {
        own = units_of(threadIdx.x, quantum);
        const int64_t first = block_scan(own, from);
        if (seqs <= Cfg::NUM_THREADS)
            return first;
        int64_t mine = 0, ahead;
        for (int s = threadIdx.x + Cfg::NUM_THREADS; s < seqs; s += Cfg::NUM_THREADS)
            mine += units_of(s, quantum);
        const int64_t total = first + block_scan(mine, ahead);
        block_sum = first;
        return total;
    };
    tc_fence_before_sync();
    Shares shares;
    int quantum = 1;
    shares.total = add_up(1);
    if (NT == 2 && shares.total < static_cast<int64_t>(kPagedCoarse) * gridDim.x) {
        quantum = kPagedQuantum;
        shares.total = add_up(quantum);
    }
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependents_launch();
    shares.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), shares.total));
    const bool works = static_cast<int>(blockIdx.x) < shares.ctas;
    if (threadIdx.x == 0 && p.keys == KEYS_ALL)
        p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);   // written again (after a barrier) if an item goes on
    if (works) {   // (the same answer in every thread)
        const int64_t u0 = shares.begin(blockIdx.x);
        int64_t before = 0;   // units of the sequences before this chunk
        for (int s0 = 0;; s0 += Cfg::NUM_THREADS) {
            const int s = s0 + static_cast<int>(threadIdx.x);
            if (own > 0 && before + from <= u0 && u0 < before + from + own) {   // one thread: unit u0 is in its sequence
                const int64_t at = u0 - before - from;
                start.s = s;
                start.q = seq_items<Cfg>(p, s);
                const int64_t per_head = own / p.kv_heads;
                start.head = static_cast<int>(at / per_head);
                start_at = at - start.head * per_head;
                start.tile = 0;
                start.unit = start.q.tiles > 1 ? 0 : static_cast<int>(start_at);
                start.quantum = quantum;
                start.left = shares.begin(blockIdx.x + 1) - u0;
            }
            before += block_sum;
            if (s0 + Cfg::NUM_THREADS >= seqs || before > u0)
                break;
            own = units_of(s + Cfg::NUM_THREADS, quantum);
            block_scan(own, from);
        }
        __syncthreads();
        // the tile that holds it
        const Walk w = start;
        if (w.q.tiles > 1) {
            locate_tile<Cfg>(w.q, quantum, start_at, static_cast<int>(threadIdx.x), Cfg::NUM_THREADS, block_scan, [&](int t, int unit) {
                start.tile = t;
                start.unit = unit;
            });
            __syncthreads();
        }
    }
    Walk walk = {};
    if (works)
        walk = start;
    const WaitCtl wc{abort_flag, p.err, p.timeout_ns};

    if (!works) {
        // fewer units than CTAs
    } else if (warp == Cfg::PRODUCER_WARP) {
        // ---------------------------------------------------------------- TMA producer
        // Lane i fetches the page number of page i of a block and, with the others, issues the
        // boxes of its K and V tiles.
        const int page_rows = 1 << p.batch.page_shift;
        const int box_rows = min(page_rows, BKV), boxes = BKV / box_rows;   // boxes per atom of a tile
        RingPos<STAGES> pos;
        uint32_t issued = 0, issued_parity = 0, q_issued = 0, q_issued_parity = 0;
        QueryPos qp(NT == 1 ? p.q_bufs : 1);
        bool ok = true;
        Segment g;
        while (ok && next_segment<Cfg>(p, walk, g)) {
            // the scores that read this buffer before are complete
            if (!(ok = wait_warp(bar.q_empty0 + 8u * qp.buf, qp.parity ^ 1u, wc, ERR_PRODUCER_SLOT, lane)))
                break;
            const uint32_t q_full = bar.q_full0 + 8u * qp.buf;
            if (lane == 0)
                mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(NT * ATOMS * g.tile_tokens * p.group * 128));
            __syncwarp();
            if (lane < NT * ATOMS) {
                const int t = lane / ATOMS, a = lane % ATOMS;
                const int at = NT == 1 ? (qp.buf * ATOMS + a) * p.q_rows * 128 : t * Cfg::Q_TILE + a * Cfg::Q_ATOM;
                tma_load_4d(sQ + static_cast<uint32_t>(at), g.prefix ? &tmap_qp : &tmap_q, q_full, 64 * a, 0, g.head,
                            g.tok0 + g.tile_first<NT>(t));
            }
            q_issued |= 1u << qp.buf;
            q_issued_parity = (q_issued_parity & ~(1u << qp.buf)) | (qp.parity << qp.buf);
            qp.step();
            // pages of this stretch: numbers past the last key's page (and bad ones) become
            // num_pages, which TMA reads as zeros
            const int key_base = g.prefix || p.keys == KEYS_ALL ? 0 : p.batch.prefix_len;
            const int own_pages = (g.kv + page_rows - 1) >> p.batch.page_shift;
            auto page_of = [&](int b) -> int {
                if (lane >= boxes || b >= g.b1)
                    return 0;
                const int lp = (key_base + b * BKV + lane * box_rows) >> p.batch.page_shift;
                int id;
                if (lp < p.n_prefix_pages)
                    id = __ldg(p.prefix_pages + lp);
                else if (!g.prefix && lp - p.n_prefix_pages < own_pages)
                    id = __ldg(p.batch.table + g.s * p.batch.table_stride + (lp - p.n_prefix_pages));
                else
                    return p.batch.num_pages;
                if (id < 0 || id >= p.batch.num_pages) {
                    atomicCAS(p.err, 0u, static_cast<uint32_t>(ERR_BATCH_INDEX));
                    id = p.batch.num_pages;
                }
                return id;
            };
            int id_next = page_of(g.b0);
            for (int b = g.b0; ok && b < g.b1; ++b) {
                const int id = id_next;
                id_next = page_of(b + 1);
                const int box = lane % boxes, atom = lane / boxes;
                const int page = __shfl_sync(0xffffffffu, id, box);
                const int row = (key_base + b * BKV) & (page_rows - 1);   // 0 unless a page holds several blocks
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!wait_warp(bar.empty0 + 8u * pos.slot, pos.parity ^ 1u, wc, ERR_PRODUCER_SLOT, lane)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = bar.full0 + 8u * pos.slot;
                    if ((p.debug & DEBUG_WITHHOLD_FIRST_LOAD) && issued == 0) {   // test hook: never loaded
                        ok = false;
                        break;
                    }
                    if (lane == 0)
                        mbar_arrive_expect_tx(fb, Cfg::KV_TILE);
                    __syncwarp();
                    if (lane < boxes * ATOMS)
                        tma_load_4d(ring + static_cast<uint32_t>(pos.slot * Cfg::KV_TILE + atom * Cfg::KV_ATOM + box * box_rows * 128),
                                    kv == 0 ? &tmap_k : &tmap_v, fb, 64 * atom, row, g.head, page);
                    issued |= 1u << pos.slot;
                    issued_parity = (issued_parity & ~(1u << pos.slot)) | (pos.parity << pos.slot);
                    pos.step();
                }
            }
        }
        if (!ok && lane == 0) {   // let every copy this warp started land before the CTA exits
            for (int i = 0; i < Cfg::Q_BUFS; ++i)
                if (q_issued & (1u << i))
                    wait_until(bar.q_full0 + 8u * i, (q_issued_parity >> i) & 1u, p.timeout_ns, p.err);
            for (int s = 0; s < STAGES; ++s)
                if (issued & (1u << s))
                    wait_until(bar.full0 + 8u * s, (issued_parity >> s) & 1u, p.timeout_ns, p.err);
        }
        __syncwarp();
    } else if (warp == Cfg::MMA_WARP) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            // descriptors: Q and K K-major (atoms of 64 dims, 32 bytes per 16), V MN-major (atoms of
            // 64 dims apart by KV_ATOM, 16 keys per 2048 bytes)
            const uint64_t q_desc = sw128_desc(sQ, 16, 1024), k_desc = sw128_desc(ring, 16, 1024);
            const uint64_t v_desc = sw128_desc(ring, Cfg::KV_ATOM, 1024);
            // (NT = 1: a query buffer holds q_rows rows per atom; the tile's other rows read on into
            // whatever follows, within the ring at most, and their scores are not used)
            const int q_atom = NT == 1 ? p.q_rows * 128 : Cfg::Q_ATOM;
            auto issue_s = [&](int t, int slot, uint32_t d) {   // S = Q_t K^T (t: tile, or query buffer)
                const uint64_t qd = q_desc + static_cast<uint64_t>((t * ATOMS * q_atom) >> 4);
                const uint64_t kd = k_desc + static_cast<uint64_t>((slot * Cfg::KV_TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < Cfg::D / 16; ++kk) {
                    const uint64_t qo = static_cast<uint64_t>(((kk >> 2) * q_atom + (kk & 3) * 32) >> 4);
                    const uint64_t ko = static_cast<uint64_t>(((kk >> 2) * Cfg::KV_ATOM + (kk & 3) * 32) >> 4);
                    umma_f16<1>(d, qd + qo, kd + ko, Cfg::ID_S, kk != 0 ? 1u : 0u);
                }
            };
            auto issue_pv = [&](int slot, uint32_t a, uint32_t d, int k0, int k1, bool add) {   // O += P V, 16-key steps
                const uint64_t vd = v_desc + static_cast<uint64_t>((slot * Cfg::KV_TILE) >> 4);
#pragma unroll
                for (int kk = k0; kk < k1; ++kk)
                    umma_f16_tmem_a(d, a + 8u * static_cast<uint32_t>(kk), vd + static_cast<uint64_t>(kk * (2048 >> 4)), Cfg::ID_PV,
                                    add || kk > 0 ? 1u : 0u);
            };
            bool ok = true;
            QueryPos qp(NT == 1 ? p.q_bufs : 1);   // of the next item (or, within one, behind this one's)
            if constexpr (NT == 1) {
                // One tile, score buffers taken in turn: the scores of the next block are issued
                // ahead of this block's product, those of a new item only if its queries are here.
                Walk ahead = walk;
                Segment gs, gp;
                RingPos<STAGES> ks, kp;          // K tile of the next scores, of the next product
                RingPos<STAGES> freed;           // V tile of the product two blocks back
                uint32_t ns = 0, np = 0;         // blocks whose scores / products are issued
                bool more_s = next_segment<Cfg>(p, ahead, gs), more_p = next_segment<Cfg>(p, walk, gp);
                int bs = gs.b0, bp = gp.b0;
                freed.step();
                int q_buf = 0;                   // of the item whose scores are being issued
                auto scores = [&]() -> bool {
                    if (bs == gs.b0) {
                        if (!wait_bounded(bar.q_full0 + 8u * qp.buf, qp.parity, wc, ERR_MMA_OPERANDS))
                            return false;
                        q_buf = qp.buf;
                        qp.step();
                    }
                    if (!wait_bounded(bar.full0 + 8u * ks.slot, ks.parity, wc, ERR_MMA_OPERANDS))
                        return false;
                    if (ns >= 2) {   // this buffer's P has been multiplied
                        if (!wait_bounded(bar.empty0 + 8u * freed.slot, freed.parity, wc, ERR_MMA_ACCUMULATOR))
                            return false;
                        freed.step();
                        freed.step();
                    }
                    tc_fence_after_sync();
                    issue_s(q_buf, ks.slot, tmem + static_cast<uint32_t>(Cfg::S_COL + static_cast<int>(ns & 1u) * BKV));
                    umma_commit(bar.empty0 + 8u * ks.slot);   // K read, scores complete
                    if (bs + 1 == gs.b1)
                        umma_commit(bar.q_empty0 + 8u * q_buf);
                    ks.step();
                    ks.step();
                    ++ns;
                    if (++bs == gs.b1) {
                        more_s = next_segment<Cfg>(p, ahead, gs);
                        bs = gs.b0;
                    }
                    return true;
                };
                auto product = [&]() -> bool {
                    RingPos<STAGES> kv = kp;
                    kv.step();
                    // (a barrier per score buffer: the softmax may finish the next block, whose
                    // scores are issued, before this thread looks)
                    if (!wait_bounded(bar.full0 + 8u * kv.slot, kv.parity, wc, ERR_MMA_OPERANDS) ||
                        !wait_bounded(bar.p_half0 + 8u * (np & 1u), (np >> 1) & 1u, wc, ERR_MMA_OPERANDS))
                        return false;
                    tc_fence_after_sync();
                    issue_pv(kv.slot, tmem + static_cast<uint32_t>(Cfg::S_COL + static_cast<int>(np & 1u) * BKV),
                             tmem + static_cast<uint32_t>(Cfg::O_COL), 0, BKV / 16, bp != gp.b0);
                    umma_commit(bar.empty0 + 8u * kv.slot);   // V read, product complete
                    kp = kv;
                    kp.step();
                    ++np;
                    if (++bp == gp.b1) {
                        more_p = next_segment<Cfg>(p, walk, gp);
                        bp = gp.b0;
                    }
                    return true;
                };
                ok = more_s && scores();
                while (ok && more_p) {
                    const bool ahead_now = more_s && (bs != gs.b0 || mbar_test_wait(bar.q_full0 + 8u * qp.buf, qp.parity));
                    if (ahead_now)
                        ok = scores();
                    ok = ok && product();
                    if (ok && !ahead_now && more_s)
                        ok = scores();
                }
            } else {
                // Two tiles share each block; as in attention_fwd_kernel: P_A V, S_A of the next
                // block, P_B V, S_B of the next block. The second tile's scores and product complete
                // the barriers that free their K and V tiles.
                RingPos<STAGES> pos;       // K tile of the current block
                uint32_t na = 0, nb = 0;   // blocks of the first and of the second tile so far
                Segment g, next;
                const uint32_t sA = tmem + static_cast<uint32_t>(Cfg::S_COL), sB = sA + BKV;
                const uint32_t oA = tmem + static_cast<uint32_t>(Cfg::O_COL), oB = oA + Cfg::D;
                bool more = next_segment<Cfg>(p, walk, next);
                while (ok && more) {
                    g = next;
                    const int mine = g.tile_blocks<NT, BKV>(0);   // the first tile's blocks
                    ok = wait_bounded(bar.q_full0, qp.parity, wc, ERR_MMA_OPERANDS);
                    qp.step();
                    auto product = [&](int t, int slot, bool add) -> bool {
                        const uint32_t n = t == 0 ? na : nb, s = t == 0 ? sA : sB, o = t == 0 ? oA : oB;
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            if (!wait_bounded((part == 0 ? bar.p_half0 : bar.p_full0) + 8u * t, n & 1u, wc, ERR_MMA_OPERANDS))
                                return false;
                            tc_fence_after_sync();
                            if (part == 0)
                                issue_pv(slot, s, o, 0, BKV / 32, add);
                            else
                                issue_pv(slot, s, o, BKV / 32, BKV / 16, true);
                        }
                        return true;
                    };
                    // scores of the block whose K tile is at `at`
                    auto scores = [&](int t, const RingPos<STAGES> &at, bool last) {
                        issue_s(t, at.slot, t == 0 ? sA : sB);
                        umma_commit(t == 0 ? bar.s_full : bar.empty0 + 8u * at.slot);
                        if (t == 1 && last)
                            umma_commit(bar.q_empty0);
                    };
                    if (ok && (ok = wait_bounded(bar.full0 + 8u * pos.slot, pos.parity, wc, ERR_MMA_OPERANDS))) {
                        tc_fence_after_sync();
                        if (g.b0 < mine)
                            scores(0, pos, false);
                        scores(1, pos, g.b0 + 1 == g.b1);
                    }
                    more = next_segment<Cfg>(p, walk, next);   // (while the softmax works)
                    for (int b = g.b0; ok && b < g.b1; ++b) {
                        RingPos<STAGES> v = pos, k_next;
                        v.step();
                        k_next = v;
                        k_next.step();
                        if (!(ok = wait_bounded(bar.full0 + 8u * v.slot, v.parity, wc, ERR_MMA_OPERANDS)))
                            break;
                        if (b < mine) {
                            if (!(ok = product(0, v.slot, b != g.b0)))
                                break;
                            umma_commit(bar.pv_done);
                            ++na;
                        }
                        if (b + 1 < g.b1) {
                            if (!(ok = wait_bounded(bar.full0 + 8u * k_next.slot, k_next.parity, wc, ERR_MMA_OPERANDS)))
                                break;
                            if (b + 1 < mine) {   // over P_A of this block
                                if (!(ok = wait_bounded(bar.pv_done, (na - 1u) & 1u, wc, ERR_MMA_ACCUMULATOR)))
                                    break;
                                tc_fence_after_sync();
                                scores(0, k_next, false);
                            }
                        }
                        if (!(ok = product(1, v.slot, b != g.b0)))
                            break;
                        umma_commit(bar.empty0 + 8u * v.slot);
                        ++nb;
                        // the next scores of this tile go over P_B (of this item's next block, or of
                        // the next item: also then P has to have been read)
                        if (!(ok = wait_bounded(bar.empty0 + 8u * v.slot, v.parity, wc, ERR_MMA_ACCUMULATOR)))
                            break;
                        tc_fence_after_sync();
                        if (b + 1 < g.b1)
                            scores(1, k_next, b + 2 == g.b1);
                        pos = k_next;
                    }
                }
            }
            if (!ok) {
                umma_commit(bar.drain);
                wait_until(bar.drain, 0, p.timeout_ns, p.err);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax
        paged_softmax_warp<Cfg>(p, bar, wc, tmem, ring, base + Cfg::STAGE_OFF + static_cast<uint32_t>(warp) * Cfg::STAGE_WARP, spoilt,
                                refs + threadIdx.x, start, shares, warp >> 2, warp, lane);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == Cfg::MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, Cfg::TMEM_COLS);
    }
}

// ---- joining the parts ---------------------------------------------------------------------------

struct CombineParams {
    int num_tokens, kv_heads, group, num_seqs;
    const int *q_start;
    int launches;
    PartsView parts[3];
    int ctas[3];                    // grid sizes of the launches
    int tile_tokens[3];
    int prefix_tokens;              // tokens per tile of prefix items
    const PartInfo *cuts[3];        // of the CTAs, or (joint) of the tokens:
    int64_t blocks[3];              // combine blocks of each launch: CTAs x blocks per item
    const PartInfo *own, *prefix;   // [num_tokens][kv_heads]
    const float *row_o[2];          // whole items of the own (0) and prefix (1) keys
    const float2 *row_ml[2];
    void *out;
    int64_t out_token, out_head;
    float *lse;
    int64_t lse_token;
};

constexpr int kCombineWarps = 8;    // per block
constexpr int kCombineRows = 32;    // rows of an item per block
// Parts up to which a warp joins four rows at once, and how many parts' loads it has in flight
// (prompts 175.4 us with 8 and 2, 178.2 with 8 and 4, 177.5 with 4 and 4).
constexpr int kCombineFew = 8, kCombineStep = 2;

struct PartAt {
    const float *o;
    const float2 *ml;
};

// A row's running sum over parts: lane's D / 32 dimensions.
template <int V>
struct RowSum {
    float m = -INFINITY, l = 0.0f;
    float acc[V] = {};
    bool sees = false;   // a part has keys for the row

    // Adds n parts, in order: lane i of a step of 32 fetches (m, l) of part i, then all lanes add up
    // their dimensions, eight parts' loads at a time. part(i): where part i's O and (m, l) are.
    template <class Part>
    __device__ __forceinline__ void add(int n, int lane, Part &&part)
    {
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int k = min(32, n - i0);
            const float2 ml = lane < k ? *part(i0 + lane).ml : make_float2(-INFINITY, 0.0f);
            float top = ml.x;
#pragma unroll
            for (int s = 16; s > 0; s /= 2)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float m_new = fmaxf(m, top);
            const float keep = m == -INFINITY ? 0.0f : exp2f(m - m_new);
            const float w = ml.y == 0.0f ? 0.0f : ml.y != ml.y ? ml.y : exp2f(ml.x - m_new);   // (NaN stays NaN)
            float sum = w * ml.y;
#pragma unroll
            for (int s = 16; s > 0; s /= 2)
                sum += __shfl_xor_sync(0xffffffffu, sum, s);
            l = l * keep + sum;
            m = m_new;
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[e] *= keep;
            const uint32_t some = __ballot_sync(0xffffffffu, !no_key(ml));
            sees = sees || some != 0;
            for (int j0 = 0; j0 < k; j0 += 8) {
                float x[8][V];
#pragma unroll
                for (int j = 0; j < 8; ++j) {   // (past the end: the last part again, with weight 0)
                    const float *src = part(i0 + min(j0 + j, k - 1)).o + lane * V;
                    if constexpr (V == 4)
                        *reinterpret_cast<float4 *>(x[j]) = *reinterpret_cast<const float4 *>(src);
                    else
                        *reinterpret_cast<float2 *>(x[j]) = *reinterpret_cast<const float2 *>(src);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool on = j0 + j < k && (some >> (j0 + j) & 1u);
                    const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        acc[e] = on ? fmaf(wj, x[j][e], acc[e]) : acc[e];
                }
            }
        }
    }

    template <typename T>
    __device__ __forceinline__ void write(const CombineParams &p, int64_t token, int head, int lane) const
    {
        const float inv = l == 0.0f ? (sees ? NAN : 0.0f) : 1.0f / l;
        T *dst = static_cast<T *>(p.out) + token * p.out_token + head * p.out_head + lane * V;
        uint32_t w[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e)
            w[e] = pack2<T>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(dst) = w[0];
        if (p.lse && lane == 0)
            p.lse[token * p.lse_token + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
};

// Joins n parts of four rows, eight lanes each (`sub`: lane of the eight), kCombineStep parts' loads
// at a time: for rows cut in few parts, of which there are many, which latency would bound otherwise.
template <typename T, int D, class Row>
__device__ __forceinline__ void combine_few(const CombineParams &p, const PartsView &v, int n, int lane, bool on, int64_t token,
                                            int head, Row &&part)
{
    constexpr int V = D / 32;   // 16-byte vectors of a lane: sub, sub + 8, ...
    const int sub = lane & 7;
    if (!on)
        return;
    float m = -INFINITY, l = 0.0f;
    float4 acc[V] = {};
    bool sees = false;   // a part has keys for the row
    for (int i0 = 0; i0 < n; i0 += kCombineStep) {
        float4 x[kCombineStep][V];
        float2 ml[kCombineStep];
#pragma unroll
        for (int i = 0; i < kCombineStep; ++i) {   // (past the end: the last part again, not counted)
            const int64_t row = part(min(i0 + i, n - 1));
            ml[i] = v.ml[row];
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[i][e] = *reinterpret_cast<const float4 *>(v.o + row * D + 4 * (sub + 8 * e));
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kCombineStep; ++i)
            top = fmaxf(top, ml[i].x);
        const float keep = m == -INFINITY ? 0.0f : exp2f(m - top);
        m = top;
        l *= keep;
#pragma unroll
        for (int e = 0; e < V; ++e)
            acc[e] = make_float4(acc[e].x * keep, acc[e].y * keep, acc[e].z * keep, acc[e].w * keep);
#pragma unroll
        for (int i = 0; i < kCombineStep; ++i) {
            if (i0 + i >= n || no_key(ml[i]))
                continue;
            sees = true;
            const float w = ml[i].y == 0.0f ? 0.0f : ml[i].y != ml[i].y ? ml[i].y : exp2f(ml[i].x - m);   // (NaN stays NaN)
            l += w * ml[i].y;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                acc[e].x = fmaf(w, x[i][e].x, acc[e].x);
                acc[e].y = fmaf(w, x[i][e].y, acc[e].y);
                acc[e].z = fmaf(w, x[i][e].z, acc[e].z);
                acc[e].w = fmaf(w, x[i][e].w, acc[e].w);
            }
        }
    }
    const float inv = l == 0.0f ? (sees ? NAN : 0.0f) : 1.0f / l;
    T *dst = static_cast<T *>(p.out) + token * p.out_token + head * p.out_head;
#pragma unroll
    for (int e = 0; e < V; ++e)
        *reinterpret_cast<uint2 *>(dst + 4 * (sub + 8 * e)) =
            make_uint2(pack2<T>(acc[e].x * inv, acc[e].y * inv), pack2<T>(acc[e].z * inv, acc[e].w * inv));
    if (p.lse && sub == 0)
        p.lse[token * p.lse_token + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over an item's parts, in the order of the keys
// (the same bits whichever CTA was first). JOINT = false: the items that CTAs left open (everything
// else is written already), kCombineRows rows per block. JOINT = true: every token and head, its
// prefix parts before its own, a warp each.
template <typename T, int D, bool JOINT>
__global__ void __launch_bounds__(32 * kCombineWarps) paged_combine_kernel(const CombineParams p)
{
    constexpr int V = D / 32;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // row of the first part (its CTA's part 1) and of the others (their CTAs' part 0)
    auto part_row = [&](const PartsView &v, int cta, int i, int tile, int r) -> int64_t {
        return (static_cast<int64_t>(2 * (cta + i) + (i == 0 ? 1 : 0)) * v.tiles + tile) * v.rows + r;
    };
    if constexpr (!JOINT) {
        int64_t at = blockIdx.x;
        int i = 0;
        while (i + 1 < p.launches && at >= p.blocks[i])
            at -= p.blocks[i++];
        const PartsView &v = p.parts[i];
        const int cta = static_cast<int>(at % p.ctas[i]), chunk = static_cast<int>(at / p.ctas[i]);
        const int4 cut = p.cuts[i][cta];
        if (cut.w < 1 || cut.w > p.ctas[i] - cta)
            return;
        const int tt = p.tile_tokens[i];
        // where an item's row is, and whether it has a token
        auto place = [&](int row, int &tile, int &r, int &tok, int &g) -> bool {
            tile = row / v.rows;
            r = row - tile * v.rows;
            tok = r / p.group;
            g = r - tok * p.group;
            const bool ok = tile < v.tiles && tok < tt && tile * tt + tok < cut.y;
            tok += tile * tt;
            return ok;
        };
        int tile, r, tok, g;
        if (cut.w <= kCombineFew) {
            const bool on = place(chunk * kCombineRows + 4 * warp + lane / 8, tile, r, tok, g);
            combine_few<T, D>(p, v, cut.w, lane, on, cut.x + tok, cut.z * p.group + g,
                              [&](int k) { return part_row(v, cta, k, tile, r); });
            return;
        }
        for (int row = chunk * kCombineRows + warp; row < (chunk + 1) * kCombineRows; row += kCombineWarps) {
            if (!place(row, tile, r, tok, g))
                continue;
            RowSum<V> sum;
            sum.add(cut.w, lane, [&](int k) {
                const int64_t at_row = part_row(v, cta, k, tile, r);
                return PartAt{v.o + at_row * D, v.ml + at_row};
            });
            sum.template write<T>(p, cut.x + tok, cut.z * p.group + g, lane);
        }
    } else {
        RowSum<V> sum;
        const int heads = p.kv_heads * p.group;
        const int64_t row = static_cast<int64_t>(blockIdx.x) * kCombineWarps + warp;
        const int64_t token = row / heads;
        const int head = static_cast<int>(row - token * heads);
        if (token >= p.num_tokens)
            return;
        const int kv_head = head / p.group, g = head - kv_head * p.group;
        const int4 info[2] = {p.own[token * p.kv_heads + kv_head], p.prefix[token * p.kv_heads + kv_head]};
        if (token < __ldg(p.q_start) || token >= __ldg(p.q_start + p.num_seqs))
            return;   // of no sequence: nothing was written for it
        int n[2], tile[2], r[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int4 &f = info[side];
            const int i = min(max(f.w, 0), p.launches - 1);
            const int tt = side == 1 ? p.prefix_tokens : p.tile_tokens[i], at = static_cast<int>(token - f.z);
            // (a token whose CTA gave up, its wait over, has no entry: what is not a possible one is left out. With
            // first tokens from 0 on, a row is among those that the parts have, also where there are fewer tokens
            // than a tile takes)
            const bool ok = f.w == i && f.y >= 1 && f.x >= 0 && f.y <= p.ctas[i] - f.x && f.z >= 0 &&
                            (f.y == 1 || (at >= 0 && at < p.parts[i].tiles * tt));
            n[side] = ok ? f.y : 0;
            tile[side] = at / tt;
            r[side] = (at - tile[side] * tt) * p.group + g;
        }
        sum.add(n[1] + n[0], lane, [&](int k) {
            const int side = k < n[1] ? 1 : 0;
            const int4 &f = info[side];
            if (f.y == 1)
                return PartAt{p.row_o[side] + row * D, p.row_ml[side] + row};
            const PartsView &v = p.parts[f.w];
            const int64_t at_row = part_row(v, f.x, side == 1 ? k : k - n[1], tile[side], r[side]);
            return PartAt{v.o + at_row * D, v.ml + at_row};
        });
        sum.template write<T>(p, token, head, lane);
    }
}

}  // namespace gb300
