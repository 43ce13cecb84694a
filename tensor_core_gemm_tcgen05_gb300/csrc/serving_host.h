// Host-side checks and launches shared by the translation units of gemm_serving.h and
// gemm_decode.h (serving_api.cu, decode_api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <limits>
#include <utility>

#include "gemm_ctx.h"
#include "gemm_serving.h"
#include "serving_common.cuh"

namespace gb300_host {

using i128 = __int128;
constexpr int64_t kMaxStride = (int64_t(1) << 39) - 8;   // elements: tensor maps hold strides below 2^40 bytes
constexpr int64_t kMaxHeads = 1 << 16;
constexpr int64_t kMaxSeqs = 1 << 24;   // (the search of a token's sequence steps past the last one in 32 bits)
constexpr int64_t kMaxKeys = (int64_t(1) << 31) - 1024;   // a block of keys may begin at the last one
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1024;   // of a batch: a tile may end past the last one

// ---- strided operands ------------------------------------------------------------------------

// Vectors of `inner` contiguous elements at base + sum_i index_i * stride_i, index_i < count_i.
struct Layout {
    const void *base;
    int64_t inner;
    int dims;
    int64_t count[3], stride[3];
};

inline int64_t span(const Layout &a)   // elements from the first to the last
{
    int64_t s = a.inner;
    for (int i = 0; i < a.dims; ++i)
        s += (a.count[i] - 1) * a.stride[i];
    return s;
}

// Sorted by stride, largest first, without the dimensions of one element.
inline Layout sorted(Layout a)
{
    int n = 0;
    for (int i = 0; i < a.dims; ++i)
        if (a.count[i] > 1) {
            a.count[n] = a.count[i];
            a.stride[n++] = a.stride[i];
        }
    a.dims = n;
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (a.stride[j] > a.stride[i]) {
                std::swap(a.stride[i], a.stride[j]);
                std::swap(a.count[i], a.count[j]);
            }
    return a;
}

// No two vectors of a (sorted) share an element: every stride covers what lies inside it.
inline bool self_disjoint(const Layout &a)
{
    int64_t s = a.inner;
    for (int i = a.dims - 1; i >= 0; --i) {
        if (a.stride[i] < s)
            return false;
        s += (a.count[i] - 1) * a.stride[i];
    }
    return true;
}

// a and b (dimension by dimension of the same strides, largest first, each covering what lies
// inside it) share no element in the dimensions i.., b moved by `delta` elements against a.
inline bool moved_disjoint(const Layout &a, const Layout &b, int i, int64_t delta)
{
    if (i == a.dims)
        return delta >= a.inner || delta <= -a.inner;
    int64_t wa = a.inner, wb = b.inner;   // width of one step of dimension i
    for (int k = i + 1; k < a.dims; ++k) {
        wa += (a.count[k] - 1) * a.stride[k];
        wb += (b.count[k] - 1) * b.stride[k];
    }
    const int64_t s = a.stride[i];
    if (delta >= wa + (a.count[i] - 1) * s || -delta >= wb + (b.count[i] - 1) * s)
        return true;
    // modulo the stride, b's steps begin at r and (the ones before) at r - s
    const int64_t r = ((delta % s) + s) % s;
    return (r >= wa || moved_disjoint(a, b, i + 1, r)) && (r - s + wb <= 0 || moved_disjoint(a, b, i + 1, r - s));
}

// a and b may share an element (both of 2-byte elements; exact where their strides agree, by
// their extents otherwise).
inline bool may_overlap(Layout a, Layout b)
{
    if (!overlaps(a.base, static_cast<size_t>(span(a)) * 2, b.base, static_cast<size_t>(span(b)) * 2))
        return false;
    if (a.dims != b.dims || a.inner != b.inner)
        return true;
    for (int i = 0; i < a.dims; ++i) {   // (the stride of a dimension of one element does not matter)
        if (a.count[i] <= 1)
            a.stride[i] = b.stride[i];
        if (b.count[i] <= 1)
            b.stride[i] = a.stride[i];
        if (a.stride[i] != b.stride[i])
            return true;
    }
    int n = 0;
    for (int i = 0; i < a.dims; ++i)
        if (a.count[i] > 1 || b.count[i] > 1) {
            a.count[n] = a.count[i];
            b.count[n] = b.count[i];
            a.stride[n] = b.stride[n] = a.stride[i];
            ++n;
        }
    a.dims = b.dims = n;
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (a.stride[j] > a.stride[i]) {
                std::swap(a.stride[i], a.stride[j]);
                std::swap(a.count[i], a.count[j]);
                std::swap(b.count[i], b.count[j]);
                b.stride[i] = a.stride[i];
                b.stride[j] = a.stride[j];
            }
    if (!self_disjoint(a) || !self_disjoint(b))
        return true;
    const int64_t bytes = static_cast<int64_t>(reinterpret_cast<intptr_t>(b.base) - reinterpret_cast<intptr_t>(a.base));
    return bytes % 2 != 0 || !moved_disjoint(a, b, 0, bytes / 2);
}

inline Layout heads_layout(const gemm_heads &h, int64_t tokens, int64_t head_dim)
{
    return Layout{h.data, head_dim, 2, {tokens, h.heads, 1}, {h.token_stride, h.head_stride, 0}};
}

inline Layout cache_layout(const gemm_kv_cache &c, const void *base)
{
    return Layout{base,
                  c.head_dim,
                  3,
                  {c.num_pages, c.kv_heads, c.page_size},
                  {c.page_stride, c.head_stride, c.row_stride}};
}

inline bool same_heads(const gemm_heads &a, const gemm_heads &b)
{
    return a.data == b.data && a.heads == b.heads && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

inline bool on_ctx(const gemm_ctx *ctx, const void *p) { return on_device(p, ctx->device); }

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Sizes, strides and alignment of one operand (not what memory it is); `out`: its vectors must
// be disjoint.
inline int check_heads(const gemm_heads *h, int64_t tokens, int64_t head_dim, bool out)
{
    if (!h || h->heads < 0 || h->heads > kMaxHeads)
        return GEMM_ERR_ARG;
    if (h->heads == 0 || tokens == 0)
        return GEMM_OK;
    if (!h->data || h->token_stride < 0 || h->head_stride < 0 || h->token_stride > kMaxStride ||
        h->head_stride > kMaxStride)
        return GEMM_ERR_ARG;
    if (static_cast<i128>(tokens) * h->token_stride + static_cast<i128>(h->heads) * h->head_stride > (i128(1) << 60))
        return GEMM_ERR_ARG;
    if (!aligned16(h->data) || h->token_stride % 8 != 0 || h->head_stride % 8 != 0)
        return GEMM_ERR_ALIGN;
    if (out && !self_disjoint(sorted(heads_layout(*h, tokens, head_dim))))
        return GEMM_ERR_ARG;
    return GEMM_OK;
}

inline int check_dtype_dim(int dtype, int64_t head_dim)
{
    return (dtype == GEMM_F16 || dtype == GEMM_BF16) && (head_dim == 64 || head_dim == 128) ? GEMM_OK : GEMM_ERR_ARG;
}

inline int check_rope(const gemm_ctx *ctx, const gemm_rope *r, int64_t head_dim)
{
    if (!r || r->rotary_dim < 0 || r->rotary_dim > head_dim || r->rotary_dim % 16 != 0 ||
        (r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->scale) || !(r->eps >= 0.0f) ||
        !std::isfinite(r->eps) || (r->rotary_dim > 0 && !r->table))
        return GEMM_ERR_ARG;
    if ((r->rotary_dim > 0 && !aligned_to(r->table, 8)) || (r->q_norm && !aligned16(r->q_norm)) ||
        (r->k_norm && !aligned16(r->k_norm)))
        return GEMM_ERR_ALIGN;
    if ((r->rotary_dim > 0 && !on_ctx(ctx, r->table)) || (r->q_norm && !on_ctx(ctx, r->q_norm)) ||
        (r->k_norm && !on_ctx(ctx, r->k_norm)))
        return GEMM_ERR_DEVICE;
    return GEMM_OK;
}

// `values`: c->v is checked too (it is not read otherwise).
inline int check_cache(const gemm_ctx *ctx, const gemm_kv_cache *c, bool values = true)
{
    if (!c || check_dtype_dim(c->dtype, c->head_dim) != GEMM_OK)
        return GEMM_ERR_ARG;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0 || c->kv_heads < 1 ||
        c->kv_heads > kMaxHeads || c->num_pages < 1 || c->num_pages > INT32_MAX - 1)
        return GEMM_ERR_ARG;
    if (!c->k || (values && !c->v) || c->page_stride <= 0 || c->head_stride <= 0 || c->row_stride <= 0 ||
        c->page_stride > kMaxStride || c->head_stride > kMaxStride || c->row_stride > kMaxStride)
        return GEMM_ERR_ARG;
    if (static_cast<i128>(c->num_pages) * c->page_stride > (i128(1) << 59))
        return GEMM_ERR_ARG;
    if (!aligned16(c->k) || (values && !aligned16(c->v)) || c->page_stride % 8 != 0 || c->head_stride % 8 != 0 ||
        c->row_stride % 8 != 0)
        return GEMM_ERR_ALIGN;
    const Layout k = cache_layout(*c, c->k), v = cache_layout(*c, c->v);
    if (!self_disjoint(sorted(k)) || (values && may_overlap(k, v)))
        return GEMM_ERR_ARG;
    if (!on_ctx(ctx, c->k) || (values && !on_ctx(ctx, c->v)))
        return GEMM_ERR_DEVICE;
    return GEMM_OK;
}

// `pointers`: the device arrays are checked too. `prefix`: prefix_pages is read.
inline int check_batch(const gemm_ctx *ctx, const gemm_kv_cache *c, const gemm_kv_batch *b, bool pointers, bool prefix)
{
    if (!b || b->num_seqs < 0 || b->num_seqs > kMaxSeqs || b->num_tokens < 0 || b->num_tokens > kMaxTokens ||
        b->max_q < 0 || b->table_width < 0 || b->table_stride < 0 || b->table_stride > kMaxStride ||
        b->num_prefix_pages < 0)
        return GEMM_ERR_ARG;
    if (b->table_width > INT32_MAX || b->num_prefix_pages > INT32_MAX ||
        (b->table_width + b->num_prefix_pages) * c->page_size > kMaxKeys)
        return GEMM_ERR_ARG;
    if (!pointers || b->num_seqs == 0 || b->num_tokens == 0)
        return GEMM_OK;
    const bool table = b->table_width > 0, pre = prefix && b->num_prefix_pages > 0;
    if (!b->q_start || !b->kv_lens || (table && !b->page_table) || (pre && !b->prefix_pages))
        return GEMM_ERR_ARG;
    if (!aligned_to(b->q_start, 4) || !aligned_to(b->kv_lens, 4) || (table && !aligned_to(b->page_table, 4)) ||
        (pre && !aligned_to(b->prefix_pages, 4)))
        return GEMM_ERR_ALIGN;
    if (!on_ctx(ctx, b->q_start) || !on_ctx(ctx, b->kv_lens) || (table && !on_ctx(ctx, b->page_table)) ||
        (pre && !on_ctx(ctx, b->prefix_pages)))
        return GEMM_ERR_DEVICE;
    return GEMM_OK;
}

inline gb300::BatchView batch_view(const gemm_kv_cache &c, const gemm_kv_batch &b)
{
    gb300::BatchView v;
    v.q_start = b.q_start;
    v.kv_lens = b.kv_lens;
    v.table = b.page_table;
    v.table_stride = b.table_stride;
    v.num_seqs = static_cast<int>(b.num_seqs);
    v.num_tokens = static_cast<int>(b.num_tokens);
    v.table_width = static_cast<int>(b.table_width);
    v.num_pages = static_cast<int>(c.num_pages);
    v.page_shift = 0;
    while ((int64_t(1) << v.page_shift) < c.page_size)
        ++v.page_shift;
    v.prefix_len = static_cast<int>(b.num_prefix_pages * c.page_size);
    return v;
}

// scale * log2(e). 0 becomes the smallest number of its sign, so that -inf times it stays -inf: finite scores times 2^-149
// are below 2^-21, less than the exponential's own error.
inline float scale_in_base_2(float scale)
{
    const float x = scale * 1.4426950408889634f;
    return x == 0.0f ? std::copysign(std::numeric_limits<float>::denorm_min(), scale) : x;
}

// Launch with programmatic stream serialisation (see gemm_api.cu): every kernel here starts with
// grid_dependency_wait.
template <typename... P, typename... A>
cudaError_t launch_serving(void (*kernel)(P...), int64_t grid, int threads, int smem, cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace gb300_host
