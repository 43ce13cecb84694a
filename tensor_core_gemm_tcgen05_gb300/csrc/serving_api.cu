// Host side of the C ABI declared in include/gemm_serving.h, and of include/gemm_decode.h's tree
// attention: argument checks, the choice of kernels and their launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>
#include <utility>

#include "gemm_ctx.h"
#include "gemm_decode.h"
#include "gemm_serving.h"
#include "paged_attention_kernel.cuh"
#include "rope_kernel.cuh"
#include "serving_host.h"

using namespace gb300_host;

namespace {

// Tiles of rows up to which prefix and own keys share a launch (32 + 8 heads of 128, 300 own keys behind 16480: one launch
// against two, 2 tiles 58 / 80 us, 4 tiles 87 / 110, 8 tiles 162 / 165, 12 tiles 236 / 221)
constexpr int64_t kJointTiles = 4;

// ---- rotation ---------------------------------------------------------------------------------

gb300::HeadsView heads_view(const gemm_heads &in, const gemm_heads &out)
{
    return gb300::HeadsView{in.data, in.token_stride, in.head_stride, out.data, out.token_stride, out.head_stride,
                            static_cast<int>(in.heads)};
}

template <bool PAGED>
int launch_rope(gemm_ctx *ctx, int dtype, int64_t head_dim, gb300::RopeParams &p, const gemm_rope &r, cudaStream_t stream)
{
    p.table = r.table;
    p.q_norm = r.q_norm;
    p.k_norm = r.k_norm;
    p.rotary_dim = static_cast<int>(r.rotary_dim);
    p.interleaved = r.interleaved;
    p.eps = r.eps;
    p.scale = r.scale;
    p.err = ctx->d_err;
    // Up to eight heads per group of lanes (the cosines are computed once per group; with 4, 8, 16
    // and 32, ragged prompts of 6582 tokens in 32 + 8 + 8 heads take 38.6, 34.1, 37.7 and 56.9 us),
    // fewer where that leaves some of the GPU's 1024 threads per SM (at this kernel's registers) idle.
    const int64_t lanes = head_dim / 8;
    auto chunks = [](int heads, int per) { return (heads + per - 1) / per; };
    int per = 8;
    while (per > 1 && p.tokens * int64_t(chunks(p.q.heads, per) + chunks(p.k.heads, per) + chunks(p.v.heads, per)) * lanes <
                          int64_t(ctx->num_sms) * 1024)
        per /= 2;
    p.heads_per_item = per;
    p.q_chunks = chunks(p.q.heads, per);
    p.k_chunks = chunks(p.k.heads, per);
    p.chunks = p.q_chunks + p.k_chunks + chunks(p.v.heads, per);
    const int64_t per_block = gb300::kRopeThreads / lanes;
    const int64_t grid = (static_cast<int64_t>(p.tokens) * p.chunks + per_block - 1) / per_block;
    if (grid > INT32_MAX)
        return GEMM_ERR_ARG;
    DeviceGuard guard(ctx->device);
    auto run = [&](auto kernel) { return launch_serving(kernel, grid, gb300::kRopeThreads, 0, stream, p); };
    cudaError_t e;
    if (dtype == GEMM_F16)
        e = head_dim == 64 ? run(gb300::rope_kernel<__half, 64, PAGED>) : run(gb300::rope_kernel<__half, 128, PAGED>);
    else
        e = head_dim == 64 ? run(gb300::rope_kernel<__nv_bfloat16, 64, PAGED>)
                           : run(gb300::rope_kernel<__nv_bfloat16, 128, PAGED>);
    return e == cudaSuccess ? GEMM_OK : cuda_fail(ctx, e, GEMM_ERR_LAUNCH);
}

// ---- paged attention ----------------------------------------------------------------------------

// The launches of one call and where their parts of the workspace are.
struct AttnLaunch {
    int tiles = 1;            // query tiles per item (the kernel's NT)
    int64_t tile_tokens = 0, rows = 0;   // of a tile: tokens, rows kept in the workspace
    int keys = 0, seqs = 0;   // KEYS_*, SEQS_*
    int64_t grid = 0;
    int64_t o_off = 0, ml_off = 0;   // PartsView
    int64_t cuts_off = 0;
};

struct AttnPlan {
    bool empty = true, joint = false;
    int count = 0;
    AttnLaunch launch[3];
    int64_t own_off = 0, prefix_off = 0;               // PartInfo tables
    int64_t row_o_off[2] = {}, row_ml_off[2] = {};     // whole items (joint): own, prefix
    int64_t bytes = 0;
};

AttnPlan attention_plan(const gemm_ctx *ctx, const gemm_kv_cache &c, const gemm_kv_batch &b, int64_t q_heads)
{
    AttnPlan pl;
    const int64_t T = b.num_tokens, group = q_heads / c.kv_heads;
    if (T == 0 || b.num_seqs == 0 || q_heads == 0)
        return pl;
    pl.empty = false;
    const int64_t tq = 128 / group;   // tokens of a full tile
    const int64_t prefix = b.num_prefix_pages * c.page_size, own = b.table_width * c.page_size;
    const int64_t flat_tiles = (T + tq - 1) / tq;
    // The prefix by itself, for the tokens of all sequences together, when that takes fewer tiles
    // of rows than there are sequences (each of which would read the prefix again): 64 sequences of 300 keys behind
    // 2048 35.5 us against 74.3, behind 16480 58 against 449. Every row then goes through the workspace, which a short
    // prefix does not earn: behind 256 keys 30.0 against 29.3, behind 32 35 against 26 (64 of 4000 keys: 186
    // against 168 behind 256, equal at 1024; 8 of 300: equal at 4096).
    pl.joint = prefix > 0 && flat_tiles < b.num_seqs;
    auto add = [&](int tiles, int64_t tile_tokens, int keys, int seqs, int64_t max_tiles, int64_t key_count) {
        AttnLaunch &l = pl.launch[pl.count++];
        l.tiles = tiles;
        l.tile_tokens = tile_tokens;
        l.rows = std::min(tile_tokens, T) * group;
        l.keys = keys;
        l.seqs = seqs;
        const int64_t bkv = tiles == 1 ? 64 : 128;
        const int64_t units = c.kv_heads * max_tiles * std::max<int64_t>(1, (key_count + bkv - 1) / bkv);
        l.grid = std::min<int64_t>(static_cast<int64_t>(ctx->num_sms) * (tiles == 1 ? 2 : 1), units);
    };
    // Few tiles of short sequences: prefix and own keys are the items of one launch.
    const bool may_long = (b.max_q == 0 || b.max_q > tq) && T > tq;
    const bool one_launch = pl.joint && flat_tiles <= kJointTiles && !may_long;
    if (pl.joint && !one_launch)
        add(flat_tiles > 1 ? 2 : 1, tq, gb300::KEYS_PREFIX, gb300::SEQS_ALL, flat_tiles, prefix);
    const int keys = pl.joint ? gb300::KEYS_OWN : gb300::KEYS_ALL;
    const int64_t seen = own + (pl.joint ? 0 : prefix);
    // Sequences with more new tokens than a tile takes go to the two-tile kernel, the others to
    // the one-tile kernel. If max_q says that all are short the one-tile kernel takes whatever there
    // is; if they have more than a tile's on average the two-tile kernel does (a second launch for
    // a few short ones costs more than their idle rows: nine sequences of 1 to 512 tokens 145 ->
    // 115 us; 8192 tokens beside 64 single ones that see 2000 keys 553 against 558 with both, 2048 158
    // against 160, 512 behind 8000 keys 178 against 176). An unknown max_q counts as long (64 single tokens of 2000 keys 102 us,
    // 91 with max_q = 1).
    const bool may_short = !may_long || (b.num_seqs > 1 && T < b.num_seqs * tq);
    if (may_long)
        add(2, tq, keys, may_short ? gb300::SEQS_LONG : gb300::SEQS_ALL, std::min(T, T / (2 * tq) + b.num_seqs), seen);
    if (may_short) {
        // tiles no larger than the sequences need, as far as that is known: less to load per item,
        // and several query buffers in the space of one full tile
        const int64_t tt = b.max_q > 0 ? std::min(tq, b.max_q) : tq;
        add(1, tt, one_launch ? gb300::KEYS_BOTH : keys, may_long ? gb300::SEQS_SHORT : gb300::SEQS_ALL,
            std::min(T, T / tt + b.num_seqs) + (one_launch ? flat_tiles : 0), std::max(seen, prefix));
        if (one_launch)
            pl.launch[pl.count - 1].rows = std::min(tq, T) * group;
    }
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t off = at;
        at += (bytes + 255) / 256 * 256;
        return off;
    };
    if (pl.joint) {
        const int64_t info = T * c.kv_heads * static_cast<int64_t>(sizeof(gb300::PartInfo));
        pl.own_off = take(info);
        pl.prefix_off = take(info);
        for (int i = 0; i < 2; ++i) {
            pl.row_o_off[i] = take(T * q_heads * c.head_dim * 4);
            pl.row_ml_off[i] = take(T * q_heads * 8);
        }
    }
    for (int i = 0; i < pl.count; ++i) {
        const int64_t rows = 2 * pl.launch[i].grid * pl.launch[i].tiles * pl.launch[i].rows;
        pl.launch[i].o_off = take(rows * c.head_dim * 4);
        pl.launch[i].ml_off = take(rows * 8);
        pl.launch[i].cuts_off = take(pl.launch[i].grid * static_cast<int64_t>(sizeof(gb300::PartInfo)));
    }
    pl.bytes = at;
    return pl;
}

// Sizes and counts; `pointers`: the batch's device arrays too.
int check_attention(const gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, int64_t q_heads, bool pointers)
{
    if (!ctx)
        return GEMM_ERR_ARG;
    int rc = check_cache(ctx, cache);
    if (rc == GEMM_OK)
        rc = check_batch(ctx, cache, batch, pointers, true);
    if (rc != GEMM_OK)
        return rc;
    if (q_heads < 0 || q_heads > kMaxHeads || q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > 128)
        return GEMM_ERR_ARG;
    if (batch->num_tokens * q_heads > (int64_t(1) << 33))
        return GEMM_ERR_ARG;
    return GEMM_OK;
}

bool encode_4d(const gemm_ctx *ctx, CUtensorMap *map, const void *ptr, int dtype, const int64_t (&dims)[4],
               const int64_t (&strides)[3] /* elements */, const uint32_t (&box)[4])
{
    cuuint64_t d[4], s[3];
    cuuint32_t bx[4], es[4];
    for (int i = 0; i < 4; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        bx[i] = box[i];
        es[i] = 1;
    }
    for (int i = 0; i < 3; ++i)   // (that of a dimension of one element does not matter)
        s[i] = static_cast<cuuint64_t>(dims[i + 1] > 1 ? strides[i] : dims[0]) * 2;
    // L2 fetches no more than a vector: in a token-major cache the next 128 bytes are another head's,
    // and are gone again before they are wanted (200 sequences of 2000 keys, 16 heads of 64: 374 -> 297 us,
    // page-major 297 either way; heads of 128 by pieces of 128 bytes instead: 0.3 % slower)
    const CUtensorMapL2promotion l2 = dims[0] * 2 >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    return ctx->encode(map, dtype == GEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                       const_cast<void *>(ptr), d, s, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Cfg>
cudaError_t launch_paged(int64_t grid, cudaStream_t stream, const CUtensorMap &tq, const CUtensorMap &tqp,
                         const CUtensorMap &tk, const CUtensorMap &tv, const gb300::PagedParams &p)
{
    return launch_serving(gb300::paged_attention_kernel<Cfg>, grid, Cfg::NUM_THREADS, Cfg::SMEM_BYTES, stream, tq, tqp, tk, tv, p);
}

// fn(config) with the PagedConfig of these run-time choices.
template <typename T, int D, bool TREE, class Fn>
auto with_tiles(int tiles, Fn &&fn)
{
    return tiles == 1 ? fn(gb300::PagedConfig<T, D, 1, TREE>{}) : fn(gb300::PagedConfig<T, D, 2, TREE>{});
}

template <bool TREE, class Fn>
auto with_type(int dtype, int64_t head_dim, int tiles, Fn &&fn)
{
    if (dtype == GEMM_F16)
        return head_dim == 64 ? with_tiles<__half, 64, TREE>(tiles, fn) : with_tiles<__half, 128, TREE>(tiles, fn);
    return head_dim == 64 ? with_tiles<__nv_bfloat16, 64, TREE>(tiles, fn) : with_tiles<__nv_bfloat16, 128, TREE>(tiles, fn);
}

template <class Fn>
auto with_config(int dtype, int64_t head_dim, int tiles, bool tree, Fn &&fn)
{
    return tree ? with_type<true>(dtype, head_dim, tiles, fn) : with_type<false>(dtype, head_dim, tiles, fn);
}

// gemm_paged_attention, or (with a tree) gemm_tree_attention.
int run_attention(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_tree *tree,
                  const gemm_heads *q, float scale, const gemm_heads *out, float *lse, int64_t lse_stride, void *workspace,
                  int64_t workspace_bytes, void *stream)
{
    const float scale_log2 = scale_in_base_2(scale);
    if (!q || !out || !std::isfinite(scale_log2))
        return GEMM_ERR_ARG;
    int rc = check_attention(ctx, cache, batch, q->heads, true);
    if (rc != GEMM_OK)
        return rc;
    const int64_t tokens = batch->num_tokens, d = cache->head_dim;
    rc = check_heads(q, tokens, d, true);   // (no broadcast queries: a tensor map has no zero strides)
    if (rc == GEMM_OK)
        rc = check_heads(out, tokens, d, true);
    if (rc != GEMM_OK)
        return rc;
    if (out->heads != q->heads || lse_stride < 0 || lse_stride > kMaxStride)
        return GEMM_ERR_ARG;
    if (tree && (tree->mask_words < 1 || tree->mask_words > GEMM_TREE_MAX_WORDS || tree->mask_stride < 0 ||
                 tree->mask_stride > kMaxStride || static_cast<i128>(tokens) * tree->mask_stride > (i128(1) << 59)))
        return GEMM_ERR_ARG;
    const AttnPlan pl = attention_plan(ctx, *cache, *batch, q->heads);
    if (pl.empty)
        return GEMM_OK;
    if (tree && !tree->mask)
        return GEMM_ERR_ARG;
    if (tree && !aligned_to(tree->mask, 4))
        return GEMM_ERR_ALIGN;
    if (!workspace || workspace_bytes < pl.bytes || (lse && tokens > 1 && lse_stride < q->heads))
        return GEMM_ERR_ARG;
    if (!aligned_to(workspace, 256) || (lse && !aligned_to(lse, 4)))
        return GEMM_ERR_ALIGN;
    const Layout lq = heads_layout(*q, tokens, d), lo = heads_layout(*out, tokens, d);
    const Layout kc = cache_layout(*cache, cache->k), vc = cache_layout(*cache, cache->v);
    if (may_overlap(lo, lq) || may_overlap(lo, kc) || may_overlap(lo, vc))
        return GEMM_ERR_ARG;
    const size_t lse_bytes = lse ? static_cast<size_t>((tokens - 1) * lse_stride + q->heads) * 4 : 0;
    for (const Layout *l : {&lq, &lo, &kc, &vc}) {
        const size_t n = static_cast<size_t>(span(*l)) * 2;
        if (overlaps(workspace, static_cast<size_t>(pl.bytes), l->base, n) || overlaps(lse, lse_bytes, l->base, n))
            return GEMM_ERR_ARG;
    }
    if (overlaps(workspace, static_cast<size_t>(pl.bytes), lse, lse_bytes))
        return GEMM_ERR_ARG;
    if (tree) {
        const size_t n = static_cast<size_t>((tokens - 1) * tree->mask_stride + tree->mask_words) * 4;
        if (overlaps(tree->mask, n, workspace, static_cast<size_t>(pl.bytes)) || overlaps(tree->mask, n, lse, lse_bytes) ||
            overlaps(tree->mask, n, lo.base, static_cast<size_t>(span(lo)) * 2))
            return GEMM_ERR_ARG;
        if (!on_ctx(ctx, tree->mask))
            return GEMM_ERR_DEVICE;
    }
    if (!on_ctx(ctx, q->data) || !on_ctx(ctx, out->data) || !on_ctx(ctx, workspace) || (lse && !on_ctx(ctx, lse)))
        return GEMM_ERR_DEVICE;

    const int64_t group = q->heads / cache->kv_heads;
    gb300::PagedParams p = {};
    p.batch = batch_view(*cache, *batch);
    p.prefix_pages = batch->prefix_pages;
    p.n_prefix_pages = static_cast<int>(batch->num_prefix_pages);
    p.kv_heads = static_cast<int>(cache->kv_heads);
    p.group = static_cast<int>(group);
    p.long_tokens = static_cast<int>(128 / group);
    p.scale_log2 = scale_log2;
    p.out = out->data;
    p.out_token = out->token_stride;
    p.out_head = out->head_stride;
    p.lse = lse;
    p.lse_token = lse_stride;
    p.q = q->data;
    p.q_token = q->token_stride;
    p.q_head = q->head_stride;
    p.k = cache->k;
    p.v = cache->v;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.row_stride = cache->row_stride;
    if (tree) {
        p.mask = tree->mask;
        p.mask_stride = tree->mask_stride;
        p.mask_words = static_cast<int>(tree->mask_words);
    }
    p.err = ctx->d_err;
    p.timeout_ns = ctx->timeout_ns;
    p.debug = ctx->debug & GEMM_DEBUG_WITHHOLD_FIRST_LOAD;
    char *ws = static_cast<char *>(workspace);
    CUtensorMap tq, tqp, tk, tv;   // tqp: queries of prefix items, a full tile
    gb300::CombineParams cp = {};
    cp.num_tokens = static_cast<int>(tokens);
    cp.kv_heads = p.kv_heads;
    cp.group = p.group;
    cp.num_seqs = p.batch.num_seqs;
    cp.q_start = batch->q_start;
    cp.launches = pl.count;
    cp.prefix_tokens = p.long_tokens;
    cp.own = reinterpret_cast<gb300::PartInfo *>(ws + pl.own_off);
    cp.prefix = reinterpret_cast<gb300::PartInfo *>(ws + pl.prefix_off);
    for (int i = 0; i < 2; ++i) {
        cp.row_o[i] = reinterpret_cast<float *>(ws + pl.row_o_off[i]);
        cp.row_ml[i] = reinterpret_cast<float2 *>(ws + pl.row_ml_off[i]);
    }
    cp.out = p.out;
    cp.out_token = p.out_token;
    cp.out_head = p.out_head;
    cp.lse = lse;
    cp.lse_token = lse_stride;

    DeviceGuard guard(ctx->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int64_t combine_grid = 0;
    for (int i = 0; i < pl.count; ++i) {
        const AttnLaunch &l = pl.launch[i];
        p.keys = l.keys;
        p.seqs = l.seqs;
        p.launch = i;
        p.tile_tokens = static_cast<int>(l.tile_tokens);
        p.q_rows = l.keys == gb300::KEYS_BOTH ? 128 : static_cast<int>((l.tile_tokens * group + 7) / 8 * 8);
        p.busy_warps = l.keys == gb300::KEYS_BOTH ? 4 : static_cast<int>((l.tile_tokens * group + 31) / 32);
        p.q_bufs = std::min(128 / p.q_rows, gb300::PagedConfig<__half, 128, 1>::Q_BUFS);
        p.parts.o = reinterpret_cast<float *>(ws + l.o_off);
        p.parts.ml = reinterpret_cast<float2 *>(ws + l.ml_off);
        p.parts.rows = static_cast<int>(l.rows);
        p.parts.tiles = l.tiles;
        p.info[0] = reinterpret_cast<gb300::PartInfo *>(ws + pl.own_off);
        p.info[1] = reinterpret_cast<gb300::PartInfo *>(ws + pl.prefix_off);
        for (int side = 0; side < 2; ++side) {
            p.row_o[side] = reinterpret_cast<float *>(ws + pl.row_o_off[side]);
            p.row_ml[side] = reinterpret_cast<float2 *>(ws + pl.row_ml_off[side]);
        }
        p.cuts = reinterpret_cast<gb300::PartInfo *>(ws + l.cuts_off);
        cp.parts[i] = p.parts;
        cp.ctas[i] = static_cast<int>(l.grid);
        cp.tile_tokens[i] = p.tile_tokens;
        cp.cuts[i] = p.cuts;
        cp.blocks[i] = l.grid * ((l.tiles * l.rows + gb300::kCombineRows - 1) / gb300::kCombineRows);
        combine_grid += cp.blocks[i];
        const uint32_t rows = static_cast<uint32_t>(std::min<int64_t>(cache->page_size, l.tiles == 1 ? 64 : 128));
        auto encode_q = [&](CUtensorMap *map, int64_t tile_tokens) {
            return encode_4d(ctx, map, q->data, cache->dtype, {d, group, cache->kv_heads, tokens},
                             {q->head_stride, group * q->head_stride, q->token_stride},
                             {64, static_cast<uint32_t>(group), 1, static_cast<uint32_t>(tile_tokens)});
        };
        if (!encode_q(&tq, l.tile_tokens) || !encode_q(&tqp, 128 / group))
            return GEMM_ERR_LAUNCH;
        const int64_t dims[4] = {d, cache->page_size, cache->kv_heads, cache->num_pages};
        const int64_t strides[3] = {cache->row_stride, cache->head_stride, cache->page_stride};
        if (!encode_4d(ctx, &tk, cache->k, cache->dtype, dims, strides, {64, rows, 1, 1}) ||
            !encode_4d(ctx, &tv, cache->v, cache->dtype, dims, strides, {64, rows, 1, 1}))
            return GEMM_ERR_LAUNCH;
        const cudaError_t e = with_config(cache->dtype, d, l.tiles, tree != nullptr, [&](auto cfg) {
            return launch_paged<decltype(cfg)>(l.grid, st, tq, tqp, tk, tv, p);
        });
        if (e != cudaSuccess)
            return cuda_fail(ctx, e, GEMM_ERR_LAUNCH);
    }
    if (pl.joint)
        combine_grid = (tokens * q->heads + gb300::kCombineWarps - 1) / gb300::kCombineWarps;
    auto combine = [&](auto kernel) { return launch_serving(kernel, combine_grid, 32 * gb300::kCombineWarps, 0, st, cp); };
    auto by_dim = [&](auto type) {
        using T = decltype(type);
        if (pl.joint)
            return d == 64 ? combine(gb300::paged_combine_kernel<T, 64, true>) : combine(gb300::paged_combine_kernel<T, 128, true>);
        return d == 64 ? combine(gb300::paged_combine_kernel<T, 64, false>) : combine(gb300::paged_combine_kernel<T, 128, false>);
    };
    const cudaError_t e = cache->dtype == GEMM_F16 ? by_dim(__half{}) : by_dim(__nv_bfloat16{});
    return e == cudaSuccess ? GEMM_OK : cuda_fail(ctx, e, GEMM_ERR_LAUNCH);
}

}  // namespace

namespace gb300_host {

cudaError_t serving_init(gemm_ctx *)
{
    for (int dtype : {GEMM_F16, GEMM_BF16})
        for (int d : {64, 128})
            for (int tiles : {1, 2})
                for (bool tree : {false, true}) {
                    const cudaError_t e = with_config(dtype, d, tiles, tree, [](auto cfg) {
                        using Cfg = decltype(cfg);
                        return cudaFuncSetAttribute(gb300::paged_attention_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    Cfg::SMEM_BYTES);
                    });
                    if (e != cudaSuccess)
                        return e;
                }
    return cudaSuccess;
}

}  // namespace gb300_host

extern "C" {

int gemm_rope_table(int64_t rotary_dim, double base, int scaling, double factor, double original, uint64_t *table,
                    float *scale)
{
    if (!table || rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0 || !(base > 1.0) || !std::isfinite(base) ||
        scaling < GEMM_ROPE_PLAIN || scaling > GEMM_ROPE_YARN || !(factor >= 1.0) || !std::isfinite(factor))
        return GEMM_ERR_ARG;
    if (scaling == GEMM_ROPE_YARN && (!(original > 0.0) || !std::isfinite(original)))
        return GEMM_ERR_ARG;
    const double two_pi = 6.283185307179586476925;
    const int64_t half = rotary_dim / 2;
    if (scaling == GEMM_ROPE_NTK)
        base *= std::pow(factor, static_cast<double>(rotary_dim) / static_cast<double>(rotary_dim - 2));
    for (int64_t i = 0; i < half; ++i) {
        double f = std::pow(base, -static_cast<double>(i) / static_cast<double>(half));
        if (scaling == GEMM_ROPE_LINEAR)
            f /= factor;
        if (scaling == GEMM_ROPE_YARN) {
            // turns within the original length: below 1 interpolated, above 32 kept
            const double turns = original * f / two_pi;
            const double keep = std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0));
            f = keep * f + (1.0 - keep) * f / factor;
        }
        // f <= 1 rad, so under 2^62 units: fits
        table[i] = static_cast<uint64_t>(std::nearbyint(f / two_pi * 18446744073709551616.0));
    }
    if (scale)
        *scale = scaling == GEMM_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return GEMM_OK;
}

int gemm_qk_rope(gemm_ctx *ctx, int dtype, int64_t tokens, int64_t head_dim, const gemm_heads *q, const gemm_heads *k,
                 const int32_t *positions, const gemm_rope *rope, const gemm_heads *q_out, const gemm_heads *k_out,
                 void *stream)
{
    if (!ctx || tokens < 0 || tokens > INT32_MAX)
        return GEMM_ERR_ARG;
    int rc = check_dtype_dim(dtype, head_dim);
    if (rc == GEMM_OK)
        rc = check_heads(q, tokens, head_dim, false);
    if (rc == GEMM_OK)
        rc = check_heads(k, tokens, head_dim, false);
    if (rc == GEMM_OK)
        rc = check_heads(q_out, tokens, head_dim, true);
    if (rc == GEMM_OK)
        rc = check_heads(k_out, tokens, head_dim, true);
    if (rc == GEMM_OK)
        rc = check_rope(ctx, rope, head_dim);
    if (rc != GEMM_OK)
        return rc;
    if (q_out->heads != q->heads || k_out->heads != k->heads)
        return GEMM_ERR_ARG;
    if (tokens == 0 || q->heads + k->heads == 0)
        return GEMM_OK;
    if (!positions)
        return GEMM_ERR_ARG;
    if (!aligned_to(positions, 4))
        return GEMM_ERR_ALIGN;
    const gemm_heads *in[2] = {q, k}, *out[2] = {q_out, k_out};
    for (int i = 0; i < 2; ++i) {
        if (out[i]->heads == 0)
            continue;
        const Layout o = heads_layout(*out[i], tokens, head_dim);
        for (int j = 0; j < 2; ++j) {
            if (in[j]->heads > 0 && !(i == j && same_heads(*out[i], *in[i])) &&
                may_overlap(o, heads_layout(*in[j], tokens, head_dim)))
                return GEMM_ERR_ARG;
            if (i != j && out[j]->heads > 0 && may_overlap(o, heads_layout(*out[j], tokens, head_dim)))
                return GEMM_ERR_ARG;
        }
        if (overlaps(o.base, static_cast<size_t>(span(o)) * 2, positions, static_cast<size_t>(tokens) * 4))
            return GEMM_ERR_ARG;
    }
    if (!on_ctx(ctx, positions))
        return GEMM_ERR_DEVICE;
    for (int i = 0; i < 2; ++i)
        if (in[i]->heads > 0 && (!on_ctx(ctx, in[i]->data) || !on_ctx(ctx, out[i]->data)))
            return GEMM_ERR_DEVICE;
    gb300::RopeParams p = {};
    p.q = heads_view(*q, *q_out);
    p.k = heads_view(*k, *k_out);
    p.tokens = static_cast<int>(tokens);
    p.positions = positions;
    return launch_rope<false>(ctx, dtype, head_dim, p, *rope, static_cast<cudaStream_t>(stream));
}

int gemm_kv_append(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_heads *q,
                   const gemm_heads *k, const gemm_heads *v, const gemm_rope *rope, const gemm_heads *q_out, void *stream)
{
    if (!ctx)
        return GEMM_ERR_ARG;
    int rc = check_cache(ctx, cache);
    if (rc == GEMM_OK)
        rc = check_batch(ctx, cache, batch, true, false);
    if (rc != GEMM_OK)
        return rc;
    const int64_t tokens = batch->num_tokens, d = cache->head_dim;
    rc = check_heads(q, tokens, d, false);
    if (rc == GEMM_OK)
        rc = check_heads(k, tokens, d, false);
    if (rc == GEMM_OK)
        rc = check_heads(v, tokens, d, false);
    if (rc == GEMM_OK)
        rc = check_heads(q_out, tokens, d, true);
    if (rc == GEMM_OK)
        rc = check_rope(ctx, rope, d);
    if (rc != GEMM_OK)
        return rc;
    if (q_out->heads != q->heads || k->heads != cache->kv_heads || v->heads != cache->kv_heads)
        return GEMM_ERR_ARG;
    if (tokens == 0 || batch->num_seqs == 0)
        return GEMM_OK;
    const Layout kc = cache_layout(*cache, cache->k), vc = cache_layout(*cache, cache->v);
    const gemm_heads *used[4] = {q, k, v, q_out};
    for (const gemm_heads *h : used) {
        if (h->heads == 0)
            continue;
        const Layout l = heads_layout(*h, tokens, d);
        if (may_overlap(l, kc) || may_overlap(l, vc))
            return GEMM_ERR_ARG;
        if (q_out->heads > 0 && h != q_out && !(h == q && same_heads(*q, *q_out)) &&
            may_overlap(heads_layout(*q_out, tokens, d), l))
            return GEMM_ERR_ARG;
    }
    for (const gemm_heads *h : used)
        if (h->heads > 0 && !on_ctx(ctx, h->data))
            return GEMM_ERR_DEVICE;
    gb300::RopeParams p = {};
    p.q = heads_view(*q, *q_out);
    p.k = heads_view(*k, gemm_heads{cache->k, k->heads, cache->page_stride, cache->head_stride});
    p.v = heads_view(*v, gemm_heads{cache->v, v->heads, cache->page_stride, cache->head_stride});
    p.tokens = static_cast<int>(tokens);
    p.batch = batch_view(*cache, *batch);
    p.row_stride = cache->row_stride;
    return launch_rope<true>(ctx, cache->dtype, d, p, *rope, static_cast<cudaStream_t>(stream));
}

int64_t gemm_paged_attention_workspace(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, int64_t q_heads)
{
    const int rc = check_attention(ctx, cache, batch, q_heads, false);
    return rc == GEMM_OK ? attention_plan(ctx, *cache, *batch, q_heads).bytes : rc;
}

int gemm_paged_attention(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_heads *q,
                         float scale, const gemm_heads *out, float *lse, int64_t lse_stride, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    return run_attention(ctx, cache, batch, nullptr, q, scale, out, lse, lse_stride, workspace, workspace_bytes, stream);
}

int64_t gemm_tree_attention_workspace(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, int64_t q_heads)
{
    return gemm_paged_attention_workspace(ctx, cache, batch, q_heads);
}

int gemm_tree_attention(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_tree *tree,
                        const gemm_heads *q, float scale, const gemm_heads *out, float *lse, int64_t lse_stride,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!tree)
        return GEMM_ERR_ARG;
    return run_attention(ctx, cache, batch, tree, q, scale, out, lse, lse_stride, workspace, workspace_bytes, stream);
}

}  // extern "C"
