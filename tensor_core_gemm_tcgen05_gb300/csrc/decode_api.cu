// Host side of the C ABI declared in include/gemm_decode.h (tree attention apart, which shares its
// launches with paged attention in serving_api.cu): argument checks, launch shapes and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "gemm_ctx.h"
#include "gemm_decode.h"
#include "kv_upkeep_kernel.cuh"
#include "serving_host.h"
#include "w4_umma_kernel.cuh"

using namespace gb300_host;

namespace {

constexpr int64_t kMaxW4Rows = 1 << 18, kMaxW4Size = 1 << 24;
constexpr int kW4SmemMax = 227 * 1024;
constexpr int kSelectHeldMax = 48 * 1024;   // keys: 192 KB of shared memory

// Which of the two 4-bit products takes up to eight rows of A: the one that these estimates (ns) give less. w4_kernel's time goes by the
// tiles of 16 rows of W and 256 columns that an SM sees and by the values of A that it lays out; w4_umma_kernel's by the
// steps of 128 x 128 an SM sees, in waves, whatever the rows. Over eight shapes from 6144 x 4096 to 65536 x 1024, groups, types and 1 to 8
// rows the choice took 0.3 % longer than the faster of both in the mean. Both sides, us (w4_kernel, the other):
//  * 1024 x 1024, eight rows, groups of 128: 3.8, 5.0; 4096 x 4096: 7.0, 8.3 (one row 6.1, 8.1); 32768 x 4096: 21.7, 33.3
//  * 16384 x 4096: one row 14.3, 16.9, eight 15.4, 17.0; groups of 64 in BF16 19.0, 19.1 and 20.1, 19.2; of 32 25.2, 23.4 and 26.5, 23.4
//  * 4096 x 16384: one row 14.8, 17.9, eight 17.8, 18.1; groups of 64 in BF16 22.6, 20.2 and 25.5, 20.3
// Of sixteen rows (of an earlier w4_kernel that took them) 16384 x 4096 took 23.2, 17.0 and 1024 x 1024 5.1, 5.1.
int64_t w4_kernel_ns(int dtype, int64_t group, int64_t tile_steps, int64_t a_steps)
{
    const int64_t per_step = dtype == GEMM_F16 ? (group == 128 ? 96 : group == 64 ? 122 : 178) : (group == 128 ? 106 : group == 64 ? 134 : 182);
    return 3400 + tile_steps * per_step + a_steps * 12;
}
int64_t w4_umma_ns(int64_t group, int64_t waves, int64_t steps)
{
    return 2400 + waves * (2900 + steps * (group == 128 ? 375 : group == 64 ? 440 : 570));
}

// launch_serving in clusters of `cluster` CTAs along x.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Bytes from the first to the last of `n` int32 (or FP32) values.
size_t words(int64_t n) { return static_cast<size_t>(std::max<int64_t>(n, 0)) * 4; }

struct Range {
    const void *base;
    size_t bytes;
};

Range range_of(const Layout &l) { return Range{l.base, static_cast<size_t>(span(l)) * 2}; }

bool overlap(const Range &a, const Range &b) { return overlaps(a.base, a.bytes, b.base, b.bytes); }

int check_seqs(const gemm_ctx *ctx, const gemm_kv_seqs *s, int64_t page_size)
{
    if (!s || s->num_seqs < 0 || s->num_seqs > kMaxSeqs || s->table_width < 0 || s->table_stride < 0 ||
        s->table_stride > kMaxStride || s->table_width > INT32_MAX || s->table_width * page_size > kMaxKeys ||
        static_cast<i128>(s->num_seqs) * s->table_stride > (i128(1) << 59))
        return GEMM_ERR_ARG;
    if (s->num_seqs == 0)
        return GEMM_OK;
    const bool table = s->table_width > 0;
    if (!s->kv_lens || (table && !s->page_table))
        return GEMM_ERR_ARG;
    if (!aligned_to(s->kv_lens, 4) || (table && !aligned_to(s->page_table, 4)))
        return GEMM_ERR_ALIGN;
    if (!on_ctx(ctx, s->kv_lens) || (table && !on_ctx(ctx, s->page_table)))
        return GEMM_ERR_DEVICE;
    return GEMM_OK;
}

Range table_range(const gemm_kv_seqs &s)
{
    return Range{s.page_table, s.table_width > 0 ? words((s.num_seqs - 1) * s.table_stride + s.table_width) : 0};
}

bool valid_pages(int64_t num_pages, int64_t page_size, int64_t kv_heads)
{
    return page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0 && kv_heads >= 1 && kv_heads <= kMaxHeads &&
           num_pages >= 1 && num_pages <= INT32_MAX - 1;
}

int check_weights(const gemm_ctx *ctx, const gemm_kv_weights *w, int64_t num_pages, int64_t page_size, int64_t kv_heads)
{
    if (!w || !w->data || w->page_stride <= 0 || w->head_stride <= 0 || w->page_stride > kMaxStride || w->head_stride > kMaxStride ||
        static_cast<i128>(num_pages) * w->page_stride > (i128(1) << 59))
        return GEMM_ERR_ARG;
    const Layout l = sorted(Layout{w->data, page_size, 2, {num_pages, kv_heads, 1}, {w->page_stride, w->head_stride, 0}});
    if (!self_disjoint(l))
        return GEMM_ERR_ARG;
    if (!aligned_to(w->data, 4))
        return GEMM_ERR_ALIGN;
    return on_ctx(ctx, w->data) ? GEMM_OK : GEMM_ERR_DEVICE;
}

Range weights_range(const gemm_kv_weights &w, int64_t num_pages, int64_t page_size, int64_t kv_heads)
{
    return Range{w.data, words((num_pages - 1) * w.page_stride + (kv_heads - 1) * w.head_stride + page_size)};
}

// Index lists [seqs][heads][most] (head_stride 0: one for all heads).
bool valid_lists(int64_t seqs, int64_t heads, int64_t most, int64_t seq_stride, int64_t head_stride, bool written)
{
    if (seq_stride < 0 || head_stride < 0 || seq_stride > kMaxStride || head_stride > kMaxStride ||
        static_cast<i128>(seqs) * seq_stride > (i128(1) << 59))
        return false;
    return !written || self_disjoint(sorted(Layout{nullptr, most, 2, {seqs, heads, 1}, {seq_stride, head_stride, 0}}));
}

int page_shift(int64_t page_size)
{
    int shift = 0;
    while ((int64_t(1) << shift) < page_size)
        ++shift;
    return shift;
}

int launched(gemm_ctx *ctx, cudaError_t e) { return e == cudaSuccess ? GEMM_OK : cuda_fail(ctx, e, GEMM_ERR_LAUNCH); }

template <typename T, class Fn>
cudaError_t with_group(int64_t group, Fn &&fn)
{
    return group == 128 ? fn(gb300::w4_kernel<T, 4>) : group == 64 ? fn(gb300::w4_kernel<T, 2>) : fn(gb300::w4_kernel<T, 1>);
}

template <class Fn>
cudaError_t with_w4(int dtype, int64_t group, Fn &&fn)
{
    return dtype == GEMM_F16 ? with_group<__half>(group, fn) : with_group<__nv_bfloat16>(group, fn);
}

template <typename T, int TOK, class Fn>
cudaError_t with_umma_group(int64_t group, Fn &&fn)
{
    return group == 128  ? fn(gb300::W4UmmaConfig<T, TOK, 128>{})
           : group == 64 ? fn(gb300::W4UmmaConfig<T, TOK, 64>{})
                         : fn(gb300::W4UmmaConfig<T, TOK, 32>{});
}

template <typename T, class Fn>
cudaError_t with_umma_tokens(int tokens, int64_t group, Fn &&fn)
{
    return tokens == 16 ? with_umma_group<T, 16>(group, fn) : tokens == 32 ? with_umma_group<T, 32>(group, fn) : with_umma_group<T, 64>(group, fn);
}

template <class Fn>
cudaError_t with_w4_umma(int dtype, int tokens, int64_t group, Fn &&fn)
{
    return dtype == GEMM_F16 ? with_umma_tokens<__half>(tokens, group, fn) : with_umma_tokens<__nv_bfloat16>(tokens, group, fn);
}

bool encode_2d(const gemm_ctx *ctx, CUtensorMap *map, CUtensorMapDataType type, int bytes, const void *ptr, int64_t cols, int64_t rows,
               int64_t stride, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride * bytes)};
    const cuuint32_t box[2] = {box_cols, box_rows}, ones[2] = {1, 1};
    return ctx->encode(map, type, 2, const_cast<void *>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace gb300_host {

cudaError_t decode_init(gemm_ctx *ctx)
{
    for (int dtype : {GEMM_F16, GEMM_BF16})
        for (int64_t group : {32, 64, 128}) {
            const cudaError_t e = with_w4(dtype, group, [&](auto kernel) {
                return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4SmemMax);
            });
            if (e != cudaSuccess)
                return e;
        }
    for (int dtype : {GEMM_F16, GEMM_BF16})
        for (int tokens : {16, 32, 64})
            for (int64_t group : {32, 64, 128}) {
                const cudaError_t e = with_w4_umma(dtype, tokens, group, [&](auto cfg) {
                    using Cfg = decltype(cfg);
                    return cudaFuncSetAttribute(gb300::w4_umma_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
                });
                if (e != cudaSuccess)
                    return e;
            }
    // clusters of the 4-bit product that run at once, a CTA to an SM
    ctx->w4_clusters[1] = ctx->num_sms;
    for (int size : {2, 4, 8}) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(size));
        cfg.blockDim = dim3(gb300::kW4Threads);
        cfg.dynamicSmemBytes = kW4SmemMax;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(size);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&ctx->w4_clusters[size], gb300::w4_kernel<__half, 4>, &cfg);
        if (e != cudaSuccess)
            return e;
    }
    return cudaFuncSetAttribute(gb300::kv_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectHeldMax * 4);
}

}  // namespace gb300_host

extern "C" {

int gemm_tree_mask(gemm_ctx *ctx, const gemm_kv_batch *batch, int64_t prefix_len, const int32_t *parents, uint32_t *mask,
                   int64_t mask_words, int64_t mask_stride, int32_t *positions, void *stream)
{
    if (!ctx || !batch || batch->num_seqs < 0 || batch->num_seqs > kMaxSeqs || batch->num_tokens < 0 ||
        batch->num_tokens > kMaxTokens || prefix_len < 0 || prefix_len > kMaxKeys || mask_words < 1 ||
        mask_words > GEMM_TREE_MAX_WORDS || mask_stride < 0 || mask_stride > kMaxStride ||
        static_cast<i128>(batch->num_tokens) * mask_stride > (i128(1) << 59))
        return GEMM_ERR_ARG;
    const int64_t tokens = batch->num_tokens;
    if (tokens == 0 || batch->num_seqs == 0)
        return GEMM_OK;
    if (!batch->q_start || !batch->kv_lens || !parents || !mask || (tokens > 1 && mask_stride < mask_words))
        return GEMM_ERR_ARG;
    const Range in[3] = {{batch->q_start, words(batch->num_seqs + 1)}, {batch->kv_lens, words(batch->num_seqs)}, {parents, words(tokens)}};
    const Range out[2] = {{mask, words((tokens - 1) * mask_stride + mask_words)}, {positions, positions ? words(tokens) : 0}};
    for (const Range &r : in)
        if (!aligned_to(r.base, 4))
            return GEMM_ERR_ALIGN;
    for (const Range &r : out)
        if (!aligned_to(r.base, 4))
            return GEMM_ERR_ALIGN;
    if (overlap(out[0], out[1]))
        return GEMM_ERR_ARG;
    for (const Range &r : in)
        if (overlap(out[0], r) || overlap(out[1], r))
            return GEMM_ERR_ARG;
    for (const Range &r : in)
        if (!on_ctx(ctx, r.base))
            return GEMM_ERR_DEVICE;
    if (!on_ctx(ctx, mask) || (positions && !on_ctx(ctx, positions)))
        return GEMM_ERR_DEVICE;
    gb300::TreeMaskParams p = {};
    p.q_start = batch->q_start;
    p.kv_lens = batch->kv_lens;
    p.parents = parents;
    p.num_tokens = static_cast<int>(tokens);
    p.prefix_len = static_cast<int>(prefix_len);
    p.mask = mask;
    p.mask_stride = mask_stride;
    p.mask_words = static_cast<int>(mask_words);
    p.positions = positions;
    p.err = ctx->d_err;
    DeviceGuard guard(ctx->device);
    return launched(ctx, launch_serving(gb300::tree_mask_kernel, batch->num_seqs, gb300::kTreeThreads, 0,
                                        static_cast<cudaStream_t>(stream), p));
}

int gemm_kv_weigh(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_heads *q, float scale,
                  const float *lse, int64_t lse_stride, int64_t window, float decay, const gemm_kv_weights *weights,
                  void *stream)
{
    const float scale_log2 = scale_in_base_2(scale);
    if (!ctx || !cache || !q || !std::isfinite(scale_log2) || !(decay >= 0.0f && decay <= 1.0f) || window < 0 || lse_stride < 0 ||
        lse_stride > kMaxStride || (batch && static_cast<i128>(batch->num_tokens) * lse_stride > (i128(1) << 59)))
        return GEMM_ERR_ARG;
    int rc = check_cache(ctx, cache, false);
    if (rc == GEMM_OK)
        rc = check_batch(ctx, cache, batch, true, false);
    if (rc == GEMM_OK)
        rc = check_heads(q, batch->num_tokens, cache->head_dim, false);
    if (rc != GEMM_OK)
        return rc;
    const int64_t tokens = batch->num_tokens, heads = cache->kv_heads, group = q->heads / heads;
    if (q->heads < heads || q->heads % heads != 0 || group > 128 || tokens * group > kMaxTokens)
        return GEMM_ERR_ARG;
    rc = check_weights(ctx, weights, cache->num_pages, cache->page_size, heads);
    if (rc != GEMM_OK)
        return rc;
    if (batch->num_seqs == 0 || tokens == 0)
        return GEMM_OK;
    if (!lse || (tokens > 1 && lse_stride < q->heads))
        return GEMM_ERR_ARG;
    if (!aligned_to(lse, 4))
        return GEMM_ERR_ALIGN;
    const Range out = weights_range(*weights, cache->num_pages, cache->page_size, heads);
    const Layout kc = cache_layout(*cache, cache->k), lq = heads_layout(*q, tokens, cache->head_dim);
    const gemm_kv_seqs seqs = {batch->num_seqs, batch->kv_lens, batch->page_table, batch->table_width, batch->table_stride};
    if (overlap(out, range_of(kc)) || overlap(out, range_of(lq)) || overlap(out, {lse, words((tokens - 1) * lse_stride + q->heads)}) ||
        overlap(out, {batch->q_start, words(batch->num_seqs + 1)}) || overlap(out, {batch->kv_lens, words(batch->num_seqs)}) ||
        overlap(out, table_range(seqs)))
        return GEMM_ERR_ARG;
    if (!on_ctx(ctx, q->data) || !on_ctx(ctx, lse))
        return GEMM_ERR_DEVICE;
    gb300::WeighParams p = {};
    p.batch = batch_view(*cache, *batch);
    p.q = q->data;
    p.q_token = q->token_stride;
    p.q_head = q->head_stride;
    p.k = cache->k;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.row_stride = cache->row_stride;
    p.lse = lse;
    p.lse_token = lse_stride;
    p.w = weights->data;
    p.w_page = weights->page_stride;
    p.w_head = weights->head_stride;
    p.kv_heads = static_cast<int>(heads);
    p.group = static_cast<int>(group);
    auto magic = [](int64_t x) { return static_cast<uint32_t>(((uint64_t(1) << 32) + x - 1) / x); };   // (of 1: 0, a plain division)
    p.group_magic = tokens * group <= (1 << 25) ? magic(group) : 0;
    p.heads_magic = heads <= 128 ? magic(heads) : 0;
    p.window = static_cast<int>(std::min<int64_t>(window, INT32_MAX));
    p.scale_log2 = scale_log2;
    p.decay = decay;
    p.err = ctx->d_err;
    const int64_t blocks = batch->num_seqs * heads * ((batch->table_width * cache->page_size + gb300::kWeighKeys - 1) / gb300::kWeighKeys);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(blocks, 2 * static_cast<int64_t>(ctx->num_sms)));
    DeviceGuard guard(ctx->device);
    auto run = [&](auto kernel) {
        return launch_serving(kernel, grid, gb300::kWeighThreads, 0, static_cast<cudaStream_t>(stream), p);
    };
    if (cache->dtype == GEMM_F16)
        return launched(ctx, cache->head_dim == 64 ? run(gb300::kv_weigh_kernel<__half, 64>) : run(gb300::kv_weigh_kernel<__half, 128>));
    return launched(ctx, cache->head_dim == 64 ? run(gb300::kv_weigh_kernel<__nv_bfloat16, 64>)
                                               : run(gb300::kv_weigh_kernel<__nv_bfloat16, 128>));
}

int gemm_kv_select(gemm_ctx *ctx, const gemm_kv_seqs *seqs, int64_t num_pages, int64_t page_size, int64_t kv_heads,
                   const gemm_kv_weights *weights, int64_t keep, int64_t first, int64_t recent, int32_t *index,
                   int64_t seq_stride, int64_t head_stride, int32_t *counts, void *stream)
{
    if (!ctx || !valid_pages(num_pages, page_size, kv_heads) || keep < 0 || keep > kMaxKeys || first < 0 || recent < 0 ||
        first > keep || recent > keep || first + recent > keep)
        return GEMM_ERR_ARG;
    int rc = check_seqs(ctx, seqs, page_size);
    if (rc == GEMM_OK)
        rc = check_weights(ctx, weights, num_pages, page_size, kv_heads);
    if (rc != GEMM_OK)
        return rc;
    const int64_t n = seqs->num_seqs, items = n * kv_heads;
    if (!valid_lists(n, kv_heads, keep, seq_stride, head_stride, keep > 0 && n > 0))
        return GEMM_ERR_ARG;
    if (n == 0)
        return GEMM_OK;
    if (!counts || (keep > 0 && !index))
        return GEMM_ERR_ARG;
    if (!aligned_to(counts, 4) || !aligned_to(index, 4))
        return GEMM_ERR_ALIGN;
    const Range out[2] = {{counts, words(n)}, {index, keep > 0 ? words((n - 1) * seq_stride + (kv_heads - 1) * head_stride + keep) : 0}};
    const Range in[3] = {{seqs->kv_lens, words(n)}, table_range(*seqs), weights_range(*weights, num_pages, page_size, kv_heads)};
    if (overlap(out[0], out[1]))
        return GEMM_ERR_ARG;
    for (const Range &r : in)
        if (overlap(out[0], r) || overlap(out[1], r))
            return GEMM_ERR_ARG;
    if (!on_ctx(ctx, counts) || (keep > 0 && !on_ctx(ctx, index)))
        return GEMM_ERR_DEVICE;
    gb300::SelectParams p = {};
    p.kv_lens = seqs->kv_lens;
    p.table = seqs->page_table;
    p.table_stride = seqs->table_stride;
    p.table_width = static_cast<int>(seqs->table_width);
    p.num_pages = static_cast<int>(num_pages);
    p.page_shift = page_shift(page_size);
    p.kv_heads = static_cast<int>(kv_heads);
    p.w = weights->data;
    p.w_page = weights->page_stride;
    p.w_head = weights->head_stride;
    p.keep = static_cast<int>(keep);
    p.first = static_cast<int>(first);
    p.recent = static_cast<int>(recent);
    p.index = index;
    p.seq_stride = seq_stride;
    p.head_stride = head_stride;
    p.counts = counts;
    p.err = ctx->d_err;
    // More CTAs for a long list, up to four an SM in all (fewer run at once where their keys take much shared memory) and with some thousand
    // keys each. Us with two, four and eight an SM at most, 8 heads, evictions one after the other: 12 sequences of up to 16 000 keys,
    // choice and compaction 66.6, 60.6, 60.7, the choice alone 21.5, 23.0, 23.2; 16 of up to 40 000 116, 105, 164 and 39.9, 41.3, 102; 32
    // of up to 6000 142, 146, 146 and 23.5, 27.4, 27.5. So two would be better for choices alone and short lists, four for evictions
    // of long ones. Why the pair takes longer than its parts with two is not known: with 16 sequences the compaction's CTAs, there early, are the
    // reason (116 -> 104 when they come after the choice), with 12 they are not (66.6 -> 67.3), and a single eviction of those takes 60.5 either
    // way. One sequence of 1090 keys, with a CTA's keys down to 512: 16.0 for 12.4.
    const int64_t room = seqs->table_width * page_size;
    int cluster = 1;
    while (cluster < 8 && items * cluster * 2 <= 4 * static_cast<int64_t>(ctx->num_sms) && room >= 4096 * cluster)
        cluster *= 2;
    if (items * cluster > INT32_MAX)
        return GEMM_ERR_ARG;
    p.held = static_cast<int>(std::min<int64_t>(kSelectHeldMax, ((room + cluster - 1) / cluster + 16 + 3) / 4 * 4));
    DeviceGuard guard(ctx->device);
    return launched(ctx, launch_cluster(gb300::kv_select_kernel, dim3(static_cast<unsigned>(items * cluster)), gb300::kSelectThreads,
                                        p.held * 4, cluster, static_cast<cudaStream_t>(stream), p));
}

int gemm_kv_compact(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_seqs *seqs, const gemm_kv_weights *weights,
                    const int32_t *index, int64_t seq_stride, int64_t head_stride, int64_t most, const int32_t *start,
                    const int32_t *counts, int32_t *new_lens, void *stream)
{
    if (!ctx || most < 0 || most > kMaxKeys)
        return GEMM_ERR_ARG;
    int rc = check_cache(ctx, cache);
    if (rc == GEMM_OK)
        rc = check_seqs(ctx, seqs, cache->page_size);
    if (rc == GEMM_OK && weights)
        rc = check_weights(ctx, weights, cache->num_pages, cache->page_size, cache->kv_heads);
    if (rc != GEMM_OK)
        return rc;
    const int64_t n = seqs->num_seqs, heads = cache->kv_heads;
    if (!valid_lists(n, heads, most, seq_stride, head_stride, false))
        return GEMM_ERR_ARG;
    if (n == 0)
        return GEMM_OK;
    if (!counts || (most > 0 && !index))
        return GEMM_ERR_ARG;
    if (!aligned_to(counts, 4) || !aligned_to(index, 4) || !aligned_to(start, 4) || !aligned_to(new_lens, 4))
        return GEMM_ERR_ALIGN;
    const Range w = weights ? weights_range(*weights, cache->num_pages, cache->page_size, heads) : Range{nullptr, 0};
    const Range out[4] = {range_of(cache_layout(*cache, cache->k)), range_of(cache_layout(*cache, cache->v)), w,
                          {new_lens, new_lens ? words(n) : 0}};
    const Range in[5] = {{seqs->kv_lens, words(n)},
                         table_range(*seqs),
                         {index, most > 0 ? words((n - 1) * seq_stride + (heads - 1) * head_stride + most) : 0},
                         {start, start ? words(n) : 0},
                         {counts, words(n)}};
    for (const Range &o : out)
        for (const Range &r : in)
            if (overlap(o, r))
                return GEMM_ERR_ARG;
    for (int i = 0; i < 4; ++i)   // (keys and values may lie between each other)
        for (int j = std::max(2, i + 1); j < 4; ++j)
            if (overlap(out[i], out[j]))
                return GEMM_ERR_ARG;
    if ((most > 0 && !on_ctx(ctx, index)) || (start && !on_ctx(ctx, start)) || !on_ctx(ctx, counts) || (new_lens && !on_ctx(ctx, new_lens)))
        return GEMM_ERR_DEVICE;
    gb300::CompactParams p = {};
    p.k = cache->k;
    p.v = cache->v;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.row_stride = cache->row_stride;
    p.kv_lens = seqs->kv_lens;
    p.table = seqs->page_table;
    p.table_stride = seqs->table_stride;
    p.table_width = static_cast<int>(seqs->table_width);
    p.num_pages = static_cast<int>(cache->num_pages);
    p.page_shift = page_shift(cache->page_size);
    p.kv_heads = static_cast<int>(heads);
    if (weights) {
        p.w = weights->data;
        p.w_page = weights->page_stride;
        p.w_head = weights->head_stride;
    }
    p.index = index;
    p.seq_index = seq_stride;
    p.head_index = head_stride;
    p.most = static_cast<int>(most);
    p.start = start;
    p.counts = counts;
    p.new_lens = new_lens;
    p.err = ctx->d_err;
    // A CTA takes several heads where their rows fit its round (accepted drafts, rows in L2: 4.2 us for 200 sequences x 16 heads x 12 rows, a
    // CTA to each head 15.4); several CTAs take the rows of one head where there are more of them than fit (12 sequences x 8 heads x 2048 rows
    // 39.4 us, half as many CTAs 55.0, one to a head 66.4, twice as many 40.9).
    const int pairs = cache->head_dim == 64 ? gb300::CompactShape<64>::PAIRS : gb300::CompactShape<128>::PAIRS;
    p.heads = 1;
    while (p.heads < heads && p.heads < pairs && most * p.heads * 2 <= pairs)
        p.heads *= 2;
    p.groups = static_cast<int>((heads + p.heads - 1) / p.heads);
    const int64_t items = n * p.groups;
    int cluster = 1;
    while (cluster < 8 && items * cluster * 2 <= 4 * static_cast<int64_t>(ctx->num_sms) && most > static_cast<int64_t>(cluster) * (pairs / p.heads))
        cluster *= 2;
    if (items * cluster > INT32_MAX)
        return GEMM_ERR_ARG;
    DeviceGuard guard(ctx->device);
    auto run = [&](auto kernel) {
        return launch_cluster(kernel, dim3(static_cast<unsigned>(items * cluster)), gb300::kCompactThreads, 0, cluster,
                              static_cast<cudaStream_t>(stream), p);
    };
    return launched(ctx, cache->head_dim == 64 ? run(gb300::kv_compact_kernel<64>) : run(gb300::kv_compact_kernel<128>));
}

int gemm_w4_run(gemm_ctx *ctx, int dtype, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const gemm_w4 *w,
                const void *bias, void *C, int64_t ldc, int epilogue, void *stream)
{
    if (!ctx || !w || (dtype != GEMM_F16 && dtype != GEMM_BF16) || M < 0 || N < 0 || K < 0 || M > kMaxW4Rows || N > kMaxW4Size ||
        K > kMaxW4Size || (epilogue != GEMM_EPI_NONE && epilogue != GEMM_EPI_GELU && epilogue != GEMM_EPI_RELU) ||
        (w->group != 32 && w->group != 64 && w->group != 128) || K % w->group != 0 || lda < K || ldc < N || lda > kMaxStride || ldc > kMaxStride)
        return GEMM_ERR_ARG;
    if (N % 8 != 0 || (K > 0 && lda % 8 != 0) || ldc % 8 != 0)
        return GEMM_ERR_ALIGN;
    if (M == 0 || N == 0)
        return GEMM_OK;
    if (!C || (K > 0 && (!A || !w->codes || !w->scales)))
        return GEMM_ERR_ARG;
    if (!aligned16(C) || !aligned16(bias) || (K > 0 && (!aligned16(A) || !aligned16(w->codes) || !aligned_to(w->scales, 2))))
        return GEMM_ERR_ALIGN;
    const size_t n = static_cast<size_t>(N), k = static_cast<size_t>(K), groups = k / static_cast<size_t>(w->group);
    const Range out = {C, static_cast<size_t>((M - 1) * ldc + N) * 2};
    const Range in[5] = {{A, K > 0 ? static_cast<size_t>((M - 1) * lda + K) * 2 : 0},
                         {w->codes, n * k / 2},
                         {w->scales, n * groups * 2},
                         {w->zeros, n * groups},
                         {bias, n * 2}};
    for (const Range &r : in)
        if (overlap(out, r))
            return GEMM_ERR_ARG;
    for (const Range &r : in)
        if (r.base && r.bytes > 0 && !on_ctx(ctx, r.base))
            return GEMM_ERR_DEVICE;
    if (!on_ctx(ctx, C))
        return GEMM_ERR_DEVICE;
    gb300::W4Params p = {};
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.a = A;
    p.lda = lda;
    p.codes = w->codes;
    p.scales = w->scales;
    p.zeros = w->zeros;
    p.bias = bias;
    p.c = C;
    p.ldc = ldc;
    p.epilogue = epilogue;
    p.steps = static_cast<int>((K + 255) / 256);
    p.err = ctx->d_err;
    p.timeout_ns = ctx->timeout_ns;
    p.debug = ctx->debug & GEMM_DEBUG_WITHHOLD_FIRST_LOAD;
    // w4_kernel: A's columns have to fit the shared memory of a cluster.
    const int groups_128 = static_cast<int>(128 / w->group);
    const int64_t blocks_m = (M + gb300::kW4Rows - 1) / gb300::kW4Rows;   // (more than one only without columns: act(bias))
    p.tiles = static_cast<int>((N + 15) / 16);
    int cluster = 1;
    auto slice = [&] { return (p.steps + cluster - 1) / cluster; };
    auto fits = [&] { return gb300::w4_smem(groups_128, slice(), cluster > 1) <= kW4SmemMax; };
    while (cluster < 8 && !fits())
        cluster *= 2;
    // Fewer tiles than CTAs: the columns shared by more of them, as long as every warp has a step.
    while (cluster < 8 && int64_t(p.tiles) * cluster * 2 <= ctx->num_sms && p.steps >= 2 * cluster * gb300::kW4Warps)
        cluster *= 2;
    p.slice = slice();
    p.clusters = std::min(p.tiles, std::max(1, ctx->w4_clusters[cluster]));
    // w4_umma_kernel: as many CTAs share a tile's columns as run at once, with two steps each at least (512 x 8192, 16 rows: 8 of
    // them 7.9 us, 4 10.5; 2048 x 2048, where not all clusters of 8 run at once: 11.1, 6.2)
    const int tokens = M <= 16 ? 16 : M <= 32 ? 32 : 64, umma_steps = static_cast<int>((K + 127) / 128);
    const int64_t umma_tiles = (N + 127) / 128 * ((M + tokens - 1) / tokens);
    int umma_cluster = 1;
    while (umma_cluster < 8 && umma_tiles <= ctx->w4_clusters[umma_cluster * 2] && umma_steps >= 4 * umma_cluster)
        umma_cluster *= 2;
    const bool umma =
        K > 0 && (M > gb300::kW4Rows || !fits() ||
                  w4_umma_ns(w->group, (umma_tiles * umma_cluster + ctx->num_sms - 1) / ctx->num_sms, (umma_steps + umma_cluster - 1) / umma_cluster) <
                      w4_kernel_ns(dtype, w->group, int64_t((p.tiles + p.clusters - 1) / p.clusters) * p.slice, M * p.slice));
    DeviceGuard guard(ctx->device);
    if (umma) {
        p.steps = umma_steps;
        CUtensorMap codes, a;
        if (!encode_2d(ctx, &codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->codes, K / 2, N, K / 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_64B) ||
            !encode_2d(ctx, &a, dtype == GEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, A, K, M, lda, 64,
                       static_cast<uint32_t>(tokens), CU_TENSOR_MAP_SWIZZLE_128B))
            return GEMM_ERR_LAUNCH;
        return launched(ctx, with_w4_umma(dtype, tokens, w->group, [&](auto cfg) {
                            using Cfg = decltype(cfg);
                            return launch_cluster(gb300::w4_umma_kernel<Cfg>,
                                                  dim3(static_cast<unsigned>((N + 127) / 128 * umma_cluster),
                                                       static_cast<unsigned>((M + tokens - 1) / tokens)),
                                                  Cfg::NUM_THREADS, Cfg::SMEM_BYTES, umma_cluster, static_cast<cudaStream_t>(stream), codes, a, p);
                        }));
    }
    return launched(ctx, with_w4(dtype, w->group, [&](auto kernel) {
                        return launch_cluster(kernel, dim3(static_cast<unsigned>(p.clusters * cluster), static_cast<unsigned>(blocks_m)),
                                              gb300::kW4Threads, static_cast<int>(gb300::w4_smem(groups_128, p.slice, cluster > 1)), cluster,
                                              static_cast<cudaStream_t>(stream), p);
                    }));
}

}  // extern "C"
