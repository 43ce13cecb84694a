// What keeps a paged key/value cache in order while it is decoded from (gemm_decode.h): masks and
// positions of drafted trees, attention weight added up per key, the keys to keep chosen by it,
// and rows moved up.
#pragma once

#include "mma_sync.cuh"
#include "serving_common.cuh"

namespace gb300 {

// Words of the shared memory of a CTA of this cluster. `addr` is what mapa_shared returned, with nothing added to it. (With an
// index below zero added to a mapped address these loads faulted; since they take mapa's own results they have not.)
__device__ __forceinline__ uint2 ld_shared_cluster_u2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint4 ld_shared_cluster_u4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void report_index(uint32_t *err)
{
    atomicCAS(err, 0u, static_cast<uint32_t>(ERR_BATCH_INDEX));
}

// ---- trees -----------------------------------------------------------------------------------
//
// A node's bits are its own and those of the nodes on its way up, whose indexes fall: one walk in
// shared memory writes the words from the last to the first. A CTA per sequence; bound by the
// launch and one trip to memory: 2.0 us captured for five nodes.
constexpr int kTreeThreads = 128, kTreeMaxNodes = 2048;   // (32 * GEMM_TREE_MAX_WORDS)

struct TreeMaskParams {
    const int *q_start, *kv_lens, *parents;
    int num_tokens, prefix_len;
    uint32_t *mask;
    int64_t mask_stride;
    int mask_words;
    int *positions;
    uint32_t *err;
};

__global__ void __launch_bounds__(kTreeThreads) tree_mask_kernel(const TreeMaskParams p)
{
    __shared__ int16_t up[kTreeMaxNodes];
    grid_dependency_wait();
    grid_dependents_launch();
    const int s = blockIdx.x;
    const int raw0 = load_start(p.q_start + s), raw1 = load_start(p.q_start + s + 1), raw_kv = p.kv_lens[s];
    const int q0 = min(max(raw0, 0), p.num_tokens), n = min(max(raw1, q0), p.num_tokens) - q0, kv = max(raw_kv, 0);
    const int nodes = min(n, 32 * p.mask_words);
    bool bad = q0 != raw0 || q0 + n != raw1 || kv != raw_kv || n > kv || nodes < n || kv > INT32_MAX - 1024 - p.prefix_len;
    for (int i = threadIdx.x; i < nodes; i += kTreeThreads) {
        const int parent = p.parents[q0 + i];
        bad = bad || parent < -1 || parent >= i;
        up[i] = static_cast<int16_t>(parent < -1 || parent >= i ? -1 : parent);
    }
    if (bad)
        report_index(p.err);
    __syncthreads();
    const int base = static_cast<int>(min(static_cast<int64_t>(p.prefix_len) + max(kv - n, 0), static_cast<int64_t>(INT32_MAX - 2048)));
    for (int i = threadIdx.x; i < n; i += kTreeThreads) {
        uint32_t *row = p.mask + (q0 + i) * p.mask_stride;
        int at = i < nodes ? i : -1, above = -1;
        for (int w = p.mask_words - 1; w >= 0; --w) {
            uint32_t bits = 0;
            for (; at >= 32 * w && at >= 0; at = up[at]) {
                bits |= 1u << (at & 31);
                ++above;
            }
            row[w] = bits;
        }
        if (p.positions)
            p.positions[q0 + i] = base + max(above, 0);
    }
}

// ---- attention weight per key ------------------------------------------------------------------
//
//     w[j] = decay w[j] + sum over rows r (tokens of the window x heads of the group) of 2^(s_rj - lse_r)
//
// Keys are the rows of 16 x 8 x 16 products, 32 to a warp, loaded once straight into registers; the
// queries are the columns, brought to shared memory 64 rows at a time in the order the products
// take them. Each key's sum stays in one warp (no atomics: the same bits each time). Blocks of 256
// keys of all sequences and heads are dealt to the CTAs in turn.
//
// For a decoding token the time is the reading of K (64 sequences of 16 to 8192 keys, 8 heads of 128: 35.1 us, 0.77 of the copy rate;
// the queries through shared memory, as for more than eight rows, 35.7). For 128 rows it is the products, on 58 % of the
// tensor pipe while they run, behind 10 us of launch, lookups and first keys (5 sequences of 300 to 8200 keys 26.0, floor
// 4.6). 16 keys to a warp, three CTAs to an SM: 25.3 there, 37.2 for the token.
constexpr int kWeighThreads = 256, kWeighKeys = 256, kWeighRows = 64;

struct WeighParams {
    BatchView batch;
    const void *q, *k;
    int64_t q_token, q_head, page_stride, head_stride, row_stride;
    const float *lse;
    int64_t lse_token;
    float *w;
    int64_t w_page, w_head;
    int kv_heads, group, window;
    uint32_t group_magic, heads_magic;   // ceil(2^32 / x); 0: not used
    float scale_log2, decay;
    uint32_t *err;
};

// a / b for 0 <= a < 2^25, 0 < b <= 128 with magic = ceil(2^32 / b): the product is off by less than a 2^-32 < 1 / b. (A
// division costs about thirty instructions, the rest of a warp's 32 keys of a decoding step about three hundred.) magic = 0: any.
__device__ __forceinline__ int divide(int a, int b, uint32_t magic)
{
    return magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(a), magic)) : a / b;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWeighThreads, 2) kv_weigh_kernel(const __grid_constant__ WeighParams p)
{
    constexpr int C = D / 32;   // 16-byte pieces of a key row per lane
    __shared__ uint4 queries[2][kWeighRows * D / 8];   // of two runs of rows: [tile of 8 rows][piece][lane]
    __shared__ float minus_lse[2][kWeighRows];         // in base 2
    __shared__ int last_key[2][kWeighRows];            // that the row sees; -1: the row gives nothing
    __shared__ int64_t ahead[kWeighThreads];        // blocks up to and with each sequence of the chunk
    __shared__ int64_t warp_sum[kWeighThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int64_t before = 0;   // blocks of the chunks before
    for (int s0 = 0; s0 < p.batch.num_seqs; s0 += kWeighThreads) {
        // the blocks of this chunk's sequences
        int64_t blocks = 0;
        if (s0 + static_cast<int>(threadIdx.x) < p.batch.num_seqs) {
            const SeqView v = load_seq(p.batch, s0 + threadIdx.x);
            if (v.bad)
                report_index(p.err);
            if (v.n > 0)   // (without new tokens: as it is)
                blocks = static_cast<int64_t>((v.kv + kWeighKeys - 1) / kWeighKeys) * p.kv_heads;
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t x = __shfl_up_sync(0xffffffffu, blocks, o);
            blocks += lane >= o ? x : 0;
        }
        if (lane == 31)
            warp_sum[warp] = blocks;
        __syncthreads();
        for (int w = 0; w < warp; ++w)
            blocks += warp_sum[w];
        ahead[threadIdx.x] = blocks;
        __syncthreads();
        const int64_t total = ahead[kWeighThreads - 1];
        // this CTA's: block b of all with b mod CTAs = its number
        int64_t b = static_cast<int64_t>(blockIdx.x) - before % gridDim.x;
        b += b < 0 ? gridDim.x : 0;
        // a block, and where the warp's keys are; found while the block before it is worked on
        struct Unit {
            SeqView v;
            int head, key0;
            int page[2];   // of 16 keys each; -1: none
        };
        auto find = [&](int64_t at) {
            Unit u = {};
            if (at >= total)
                return u;
            int lo = 0;   // the first sequence with ahead > at
            for (int step = kWeighThreads / 2; step > 0; step /= 2)
                lo += ahead[lo + step - 1] <= at ? step : 0;
            u.v = load_seq(p.batch, s0 + lo);
            const int64_t in_seq = at - (lo > 0 ? ahead[lo - 1] : 0);   // block of keys by block, its heads one after the other
            const int block = in_seq < (1 << 25) ? divide(static_cast<int>(in_seq), p.kv_heads, p.heads_magic)
                                                 : static_cast<int>(in_seq / p.kv_heads);
            u.head = static_cast<int>(in_seq - static_cast<int64_t>(block) * p.kv_heads);
            u.key0 = block * kWeighKeys + 32 * warp;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int key = u.key0 + 16 * m;
                u.page[m] = key < u.v.kv ? p.batch.table[(s0 + lo) * p.batch.table_stride + (key >> p.batch.page_shift)] : -1;
            }
            return u;
        };
        Unit next = find(b);
        for (; b < total; b += gridDim.x) {
            const Unit u = next;
            const SeqView &v = u.v;
            const int head = u.head, key0 = u.key0;
            // ---- the warp's keys, and their weights before (lanes of t = 0)
            uint4 k[2][2][C];   // [tile of 16 keys][row g, g + 8][piece]
            float *weight[2];   // of key g of the tile
            float old[2][2];
            bool there[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int key = key0 + 16 * m, row = key & ((1 << p.batch.page_shift) - 1);
                there[m] = u.page[m] >= 0 && u.page[m] < p.batch.num_pages;
                if (key < v.kv && !there[m])
                    report_index(p.err);
                const T *src = static_cast<const T *>(p.k) + u.page[m] * p.page_stride + head * p.head_stride + (row + g) * p.row_stride + 8 * t;
                weight[m] = p.w + u.page[m] * p.w_page + head * p.w_head + row + g;
                old[m][0] = old[m][1] = 0.0f;
                if (there[m]) {   // (the sums of keys that are not there are not written)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            k[m][half][c] = *reinterpret_cast<const uint4 *>(src + half * 8 * p.row_stride + 32 * c);
                        if (t == 0 && p.decay != 0.0f && key + 8 * half + g < v.kv - v.n)
                            old[m][half] = weight[m][8 * half];
                    }
                }
            }
            const int tokens = p.window > 0 ? min(p.window, v.n) : v.n;
            const int rows = tokens * p.group;   // (fits: the host sees to it)
            // row r of the queries: -lse in base 2, and the last key that it sees (-1: it gives nothing)
            auto row_of = [&](int r, float &off, int &last) {
                off = 0.0f;
                last = -1;
                if (r < rows) {
                    const int token = divide(r, p.group, p.group_magic), i = v.n - tokens + token;   // of the sequence's new tokens
                    const float l = p.lse[(v.q0 + i) * p.lse_token + head * p.group + (r - token * p.group)];
                    off = -l * 1.4426950408889634f;
                    last = l == -INFINITY ? -1 : v.kv - v.n + i;
                }
            };
            auto query_at = [&](int r, int piece) {   // 8 dims of row r
                const int token = divide(r, p.group, p.group_magic);
                return reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + static_cast<int64_t>(v.q0 + v.n - tokens + token) * p.q_token +
                                                       (head * p.group + r - token * p.group) * p.q_head + 8 * piece);
            };
            float sum[2][2] = {};
            // weight of eight rows: the pieces of their queries, and of rows 2 t, 2 t + 1 the other two
            auto weigh = [&](const uint4 (&q)[C], float2 off, int2 last) {
                float s[2][4] = {};
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        mma_16x8x16<T>(s[m], k[m][0][c].x, k[m][1][c].x, k[m][0][c].y, k[m][1][c].y, q[c].x, q[c].y);
                        mma_16x8x16<T>(s[m], k[m][0][c].z, k[m][1][c].z, k[m][0][c].w, k[m][1][c].w, q[c].z, q[c].w);
                    }
                const bool all = __all_sync(0xffffffffu, min(last.x, last.y) >= key0 + 31);   // the rows see all of the warp's keys
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int key = key0 + 16 * m + 8 * half + g;
                        float x = ex2_approx(fmaf(s[m][2 * half], p.scale_log2, off.x));
                        float y = ex2_approx(fmaf(s[m][2 * half + 1], p.scale_log2, off.y));
                        if (!all) {
                            x = key <= last.x ? x : 0.0f;
                            y = key <= last.y ? y : 0.0f;
                        }
                        sum[m][half] += x + y;
                    }
            };
            if (rows <= 8) {   // (a decoding step: the queries straight into registers, no warp waits for another)
                uint4 q[C];
                float2 off;
                int2 last;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    q[c] = g < rows ? *query_at(g, 4 * c + t) : make_uint4(0, 0, 0, 0);
                row_of(2 * t, off.x, last.x);
                row_of(2 * t + 1, off.y, last.y);
                next = find(b + gridDim.x);
                weigh(q, off, last);
            } else {
                // 64 rows at a time, the next ones on their way meanwhile
                auto bring = [&](int r0, int buf) {
                    const int count = (min(rows - r0, kWeighRows) + 7) / 8 * 8;
                    for (int i = threadIdx.x; i < count * (D / 8); i += kWeighThreads) {
                        const int r = i / (D / 8), piece = i % (D / 8);
                        uint4 *dst = queries[buf] + ((r / 8) * C + piece / 4) * 32 + (r % 8) * 4 + piece % 4;
                        if (r0 + r < rows)
                            copy_async<16>(smem_u32(dst), query_at(r0 + r, piece));
                        else
                            *dst = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (threadIdx.x < static_cast<unsigned>(count))
                        row_of(r0 + threadIdx.x, minus_lse[buf][threadIdx.x], last_key[buf][threadIdx.x]);
                };
                __syncthreads();   // the rows of the block before are done with
                bring(0, 0);
                next = find(b + gridDim.x);
                for (int r0 = 0, buf = 0; r0 < rows; r0 += kWeighRows, buf ^= 1) {
                    if (r0 + kWeighRows < rows) {
                        bring(r0 + kWeighRows, buf ^ 1);
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                    } else {
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                    }
                    __syncthreads();
                    const int tiles = key0 < v.kv ? (min(rows - r0, kWeighRows) + 7) / 8 : 0;
                    for (int i = 0; i < tiles; ++i) {
                        uint4 q[C];
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            q[c] = queries[buf][(i * C + c) * 32 + lane];
                        weigh(q, *reinterpret_cast<const float2 *>(minus_lse[buf] + 8 * i + 2 * t),
                              *reinterpret_cast<const int2 *>(last_key[buf] + 8 * i + 2 * t));
                    }
                    __syncthreads();   // these rows are done with
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float x = sum[m][half];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (t == 0 && key0 + 16 * m + 8 * half + g < v.kv && there[m])
                        weight[m][8 * half] = fmaf(p.decay, old[m][half], x);
                }
        }
        before += total;
        __syncthreads();   // ahead may be written again
    }
}

// ---- choosing what to keep ---------------------------------------------------------------------
//
// The m heaviest of the keys between the first and the recent ones, exactly: the weight at the border
// is found digit by digit (11, 11 and 10 bits of an order-preserving integer), each from a histogram
// of the keys that agree with the digits before; then one pass over the keys in order writes those above the
// border and the first of those on it. A cluster of CTAs per sequence and key head, each with a
// slice of the keys, which it holds in shared memory; the histograms are summed over distributed
// shared memory. Reads each weight once. Bound by the chain of its passes, each with a barrier of the cluster: 1090 keys of 8
// heads 7.9 us, 12 sequences of 3000 to 16 000 22.9 (captured, weights from HBM).
constexpr int kSelectThreads = 512, kSelectBins = 2048, kSelectBatch = 8;

struct SelectParams {
    const int *kv_lens, *table;
    int64_t table_stride;
    int table_width, num_pages, page_shift, kv_heads;
    const float *w;
    int64_t w_page, w_head;
    int keep, first, recent;
    int *index;
    int64_t seq_stride, head_stride;
    int *counts;
    int held;   // keys of a slice that are held in shared memory
    uint32_t *err;
};

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ uint4 held_vectors[];   // (read four keys at a time: 16-byte aligned)
    uint32_t *const held = reinterpret_cast<uint32_t *>(held_vectors);
    __shared__ uint4 histograms[3][kSelectThreads];   // of each digit, the highest value first, four to a thread
    __shared__ uint32_t warp_sum[2][kSelectThreads / 32];
    __shared__ uint32_t digit, above;
    __shared__ uint2 mine;   // keys above the border, on it
    static_assert(kSelectBins == 4 * kSelectThreads, "four bins to a thread");
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
    const int item = static_cast<int>(blockIdx.x) / ctas, s = item / p.kv_heads, head = item % p.kv_heads;
    const int raw = p.kv_lens[s], kv = min(max(raw, 0), p.table_width << p.page_shift);
    if (raw != kv && threadIdx.x == 0)
        report_index(p.err);
    int *index = p.index + s * p.seq_stride + head * p.head_stride;
    const int count = min(kv, p.keep);
    if (head == 0 && rank == 0 && threadIdx.x == 0)
        p.counts[s] = count;
    for (int64_t i = count + rank * kSelectThreads + static_cast<int>(threadIdx.x); i < p.keep; i += ctas * kSelectThreads)
        index[i] = -1;
    if (kv <= p.keep) {   // (the same for all CTAs of the cluster)
        for (int64_t i = rank * kSelectThreads + static_cast<int>(threadIdx.x); i < kv; i += ctas * kSelectThreads)
            index[i] = static_cast<int>(i);
        return;
    }
    // candidates [lo, hi), of which m are kept; this CTA's keys [a, b)
    const int lo = p.first, hi = kv - p.recent, m = p.keep - p.first - p.recent;
    const int slice = static_cast<int>(((static_cast<int64_t>(kv) + ctas - 1) / ctas + 15) / 16 * 16);
    const int a = static_cast<int>(min(static_cast<int64_t>(rank) * slice, static_cast<int64_t>(kv)));
    const int b = static_cast<int>(min(static_cast<int64_t>(a) + slice, static_cast<int64_t>(kv)));
    bool bad = false;
    auto page_of = [&](int i) { return p.table[s * p.table_stride + (i >> p.page_shift)]; };
    auto weight_key = [&](int id, int i) -> uint32_t {   // of key i, whose page is id: as an integer that orders as the weights do
        // (no branch: several loads are in flight)
        const bool ok = id >= 0 && id < p.num_pages;
        bad = bad || !ok;
        float x = p.w[(ok ? id : 0) * p.w_page + head * p.w_head + (i & ((1 << p.page_shift) - 1))] + 0.0f;   // (-0 becomes 0)
        x = ok ? x : 0.0f;
        const uint32_t u = __float_as_uint(x);
        return x != x ? 0u : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
    };
    auto fetch = [&](int i) { return weight_key(page_of(i), i); };
    const int in_held = static_cast<int>(min(static_cast<int64_t>(b), static_cast<int64_t>(a) + p.held));
    auto key_of = [&](int i) -> uint32_t { return i < in_held ? held[i - a] : fetch(i); };
    if (m > 0) {   // (pages of eight keys at a time, then their weights: two trips to memory for eight)
        const int end = in_held;
        for (int i0 = a + static_cast<int>(threadIdx.x); i0 < end; i0 += kSelectBatch * kSelectThreads) {
            int id[kSelectBatch];
            uint32_t key[kSelectBatch];
#pragma unroll
            for (int e = 0; e < kSelectBatch; ++e)
                id[e] = page_of(min(i0 + e * kSelectThreads, end - 1));
#pragma unroll
            for (int e = 0; e < kSelectBatch; ++e)
                key[e] = weight_key(id[e], min(i0 + e * kSelectThreads, end - 1));
#pragma unroll
            for (int e = 0; e < kSelectBatch; ++e)
                if (i0 + e * kSelectThreads < end)
                    held[i0 + e * kSelectThreads - a] = key[e];
        }
    }
    // ---- the border
    uint32_t border = 0xffffffffu, left = 0;   // all above it (nothing is) and the first `left` on it
    if (m > 0) {
        border = 0;
        left = static_cast<uint32_t>(m);
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            uint4 *const bins = histograms[pass];   // (one for each: the other CTAs may still be reading the last)
            uint32_t *const hist = reinterpret_cast<uint32_t *>(bins);
            bins[threadIdx.x] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            auto count_digit = [&](int i, uint32_t key) {
                if (static_cast<uint32_t>(i - lo) < static_cast<uint32_t>(hi - lo) && (pass == 0 || (key ^ border) >> (shift + bits) == 0))
                    atomicAdd(&hist[(~key >> shift) & ((1u << bits) - 1u)], 1u);
            };
            for (int i = a + 4 * static_cast<int>(threadIdx.x); i < in_held; i += 4 * kSelectThreads) {   // (past the end: keys that are not counted)
                const uint4 key = *reinterpret_cast<const uint4 *>(held + (i - a));
                count_digit(i, key.x);
                count_digit(i + 1, i + 1 < in_held ? key.y : 0u);
                count_digit(i + 2, i + 2 < in_held ? key.z : 0u);
                count_digit(i + 3, i + 3 < in_held ? key.w : 0u);
            }
            for (int i = in_held + static_cast<int>(threadIdx.x); i < b; i += kSelectThreads)
                count_digit(i, fetch(i));
            __syncthreads();
            if (ctas > 1)
                cluster_sync();
            // digits from the highest down: complement 4 t + e of the low bits
            uint4 n = bins[threadIdx.x];
            for (int r = 0; r < ctas; ++r) {
                if (r == rank)
                    continue;
                const uint4 x = ld_shared_cluster_u4(mapa_shared(smem_u32(bins + threadIdx.x), static_cast<uint32_t>(r)));
                n = make_uint4(n.x + x.x, n.y + x.y, n.z + x.z, n.w + x.w);
            }
            const uint32_t sum = n.x + n.y + n.z + n.w;
            uint32_t scan = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, scan, o);
                scan += lane >= o ? x : 0;
            }
            if (lane == 31)
                warp_sum[0][warp] = scan;
            __syncthreads();
            scan -= sum;
            for (int w = 0; w < warp; ++w)
                scan += warp_sum[0][w];
            const uint32_t each[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (scan < left && left <= scan + each[e]) {   // one thread, one digit
                    digit = ~(4 * threadIdx.x + e) & ((1u << bits) - 1u);
                    above = scan;
                }
                scan += each[e];
            }
            __syncthreads();
            border |= digit << shift;
            left -= above;
        }
    }
    if (bad)
        report_index(p.err);
    // ---- how many of each kind the slices before this one have
    auto above_it = [&](int i, uint32_t key) { return i < lo || i >= hi || key > border; };
    const int piece = ((b - a + kSelectThreads - 1) / kSelectThreads) * 32;   // of the slice, to a warp
    const int wa = static_cast<int>(min(static_cast<int64_t>(a) + static_cast<int64_t>(warp) * piece, static_cast<int64_t>(b)));
    const int wb = static_cast<int>(min(static_cast<int64_t>(wa) + piece, static_cast<int64_t>(b)));
    uint32_t gt = 0, eq = 0;
    for (int i = wa + lane; i < wb; i += 32) {
        const uint32_t key = m > 0 ? key_of(i) : 0u;
        const bool up = above_it(i, key);
        gt += up;
        eq += !up && key == border;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        gt += __shfl_xor_sync(0xffffffffu, gt, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
        warp_sum[0][warp] = gt;
        warp_sum[1][warp] = eq;
    }
    __syncthreads();
    gt = eq = 0;   // of the warps before this one; thread 511: of all
    for (int w = 0; w < warp; ++w) {
        gt += warp_sum[0][w];
        eq += warp_sum[1][w];
    }
    if (ctas > 1) {
        if (threadIdx.x == kSelectThreads - 1)
            mine = make_uint2(gt + warp_sum[0][warp], eq + warp_sum[1][warp]);
        __syncthreads();
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            const uint2 x = ld_shared_cluster_u2(mapa_shared(smem_u32(&mine), static_cast<uint32_t>(r)));
            gt += x.x;
            eq += x.y;
        }
    }
    // ---- the kept keys in order, a piece of the slice per warp
    for (int i0 = wa; i0 < wb; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < wb && m > 0 ? key_of(i) : 0u;
        const bool up = i < wb && above_it(i, key), on = i < wb && !up && key == border;
        const uint32_t ups = __ballot_sync(0xffffffffu, up), ons = __ballot_sync(0xffffffffu, on), lower = (1u << lane) - 1u;
        const uint32_t g = gt + __popc(ups & lower), e = eq + __popc(ons & lower), to = g + min(e, left);
        if ((up || (on && e < left)) && to < static_cast<uint32_t>(p.keep))   // (always, unless weights change meanwhile)
            index[to] = i;
        gt += __popc(ups);
        eq += __popc(ons);
    }
    __syncthreads();
    if (ctas > 1)
        cluster_sync();   // the other CTAs have read this one's counts
}

// ---- moving rows up ------------------------------------------------------------------------------
//
// Row j <- row index[j] >= j, in order, so a round of consecutive rows j is safe once all of its own
// sources are read: sources of later rounds lie behind the rows that it writes, and those of
// earlier ones are read already. A cluster of CTAs takes a round together (loads into registers, a
// cluster barrier, stores); each CTA moves keys and values of a few heads. Bound by HBM for long lists (12 sequences x 8 heads x
// 2048 rows, 101 MB read and as much written: 39.4 us, 53 % of HBM's time busy; reads a round ahead, which took
// 117 registers, 55), by the chain of lookups for a few accepted drafts (3.9; 2.7 on rows that are in L2).
constexpr int kCompactThreads = 256, kCompactVecs = 8;   // 16-byte pieces a thread holds

struct CompactParams {
    void *k, *v;
    int64_t page_stride, head_stride, row_stride;   // elements of 2 bytes
    const int *kv_lens, *table;
    int64_t table_stride;
    int table_width, num_pages, page_shift, kv_heads;
    float *w;   // or nullptr
    int64_t w_page, w_head;
    const int *index;
    int64_t seq_index, head_index;
    int most;
    const int *start, *counts;
    int *new_lens;
    int heads, groups;   // heads of a CTA (a power of two), groups of such heads
    uint32_t *err;
};

template <int D>
struct CompactShape {
    static constexpr int PIECES = D / 8;                                          // of a row
    static constexpr int PAIRS = kCompactThreads * kCompactVecs / (2 * PIECES);   // (head, row) of a CTA's round, key and value each
};

template <int D>
__global__ void __launch_bounds__(kCompactThreads) kv_compact_kernel(const __grid_constant__ CompactParams p)
{
    using Shape = CompactShape<D>;
    constexpr int PIECES = Shape::PIECES, PAIRS = Shape::PAIRS;
    __shared__ int64_t from[2][PAIRS], to[2][PAIRS];   // elements of the cache; from < 0: not moved
    grid_dependency_wait();
    grid_dependents_launch();
    const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
    const int item = static_cast<int>(blockIdx.x) / ctas, s = item / p.groups, head0 = item % p.groups * p.heads;
    const int rows = PAIRS / p.heads;   // of each head in a CTA's round
    const int raw_kv = p.kv_lens[s], kv = min(max(raw_kv, 0), p.table_width << p.page_shift);
    const int raw_start = p.start ? p.start[s] : 0, start = min(max(raw_start, 0), kv);
    const int raw_count = p.counts[s], count = raw_start == start ? min(max(raw_count, 0), p.most) : 0;
    if (threadIdx.x == 0 && rank == 0 && head0 == 0) {
        if (raw_kv != kv || raw_start != start || raw_count < 0 || raw_count > p.most)
            report_index(p.err);
        if (p.new_lens)
            p.new_lens[s] = static_cast<int>(min(static_cast<int64_t>(start) + count, static_cast<int64_t>(INT32_MAX)));
    }
    const int mask = (1 << p.page_shift) - 1;
    const int64_t per_round = static_cast<int64_t>(ctas) * rows;
    float *weight_from = nullptr, *weight_to = nullptr;   // of the row that this thread has looked up last
    // where the rows of the round from `first` on are and go to
    auto find = [&](int64_t first, int buf) {
        if (threadIdx.x >= PAIRS)
            return;
        const int head = head0 + static_cast<int>(threadIdx.x) / rows;
        const int64_t j = first + static_cast<int64_t>(rank) * rows + static_cast<int>(threadIdx.x) % rows;
        int64_t src = -1, dst = 0;
        weight_to = nullptr;
        if (head < p.kv_heads && j < count) {
            const int i = p.index[s * p.seq_index + head * p.head_index + j];
            const int64_t row = static_cast<int64_t>(start) + i;
            if (i < j || row >= kv) {
                report_index(p.err);
            } else if (i > j) {
                const int to_row = start + static_cast<int>(j), from_row = static_cast<int>(row);
                const int *table = p.table + s * p.table_stride;
                const int a = table[from_row >> p.page_shift], b = table[to_row >> p.page_shift];
                if (a < 0 || a >= p.num_pages || b < 0 || b >= p.num_pages) {
                    report_index(p.err);
                } else {
                    src = a * p.page_stride + head * p.head_stride + (from_row & mask) * p.row_stride;
                    dst = b * p.page_stride + head * p.head_stride + (to_row & mask) * p.row_stride;
                    if (p.w) {
                        weight_from = p.w + a * p.w_page + head * p.w_head + (from_row & mask);
                        weight_to = p.w + b * p.w_page + head * p.w_head + (to_row & mask);
                    }
                }
            }
        }
        from[buf][threadIdx.x] = src;
        to[buf][threadIdx.x] = dst;
    };
    find(0, 0);
    __syncthreads();
    int buf = 0;
    for (int64_t first = 0; first < count; first += per_round, buf ^= 1) {
        // ---- read, look up the next round's rows meanwhile, wait for the others, write
        uint4 x[kCompactVecs];
#pragma unroll
        for (int e = 0; e < kCompactVecs; ++e) {
            const int at = e * kCompactThreads + static_cast<int>(threadIdx.x), row = at / PIECES, piece = at % PIECES;
            const int64_t src = from[buf][row / 2];
            const uint16_t *base = static_cast<const uint16_t *>(row % 2 ? p.v : p.k);
            if (src >= 0)
                x[e] = *reinterpret_cast<const uint4 *>(base + src + 8 * piece);
        }
        float *const store_weight = weight_to;
        const float weight = store_weight ? *weight_from : 0.0f;
        find(first + per_round, buf ^ 1);
        __syncthreads();
        if (ctas > 1)
            cluster_sync();
#pragma unroll
        for (int e = 0; e < kCompactVecs; ++e) {
            const int at = e * kCompactThreads + static_cast<int>(threadIdx.x), row = at / PIECES, piece = at % PIECES;
            uint16_t *base = static_cast<uint16_t *>(row % 2 ? p.v : p.k);
            if (from[buf][row / 2] >= 0)
                *reinterpret_cast<uint4 *>(base + to[buf][row / 2] + 8 * piece) = x[e];
        }
        if (store_weight)
            *store_weight = weight;
        __syncthreads();   // the lookups after the next go over this round's
    }
}

}  // namespace gb300
