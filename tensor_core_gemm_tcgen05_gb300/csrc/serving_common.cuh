// What the kernels of gemm_serving.h share: the two element types and the device-side view of a
// ragged batch over a paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "gemm_kernel.cuh"

namespace gb300 {

// Two values packed in 32 bits (the first in the low half), rounded to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// CTAs of this cluster (1 in a launch without clusters).
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// BYTES (4, 8 or 16) from global to shared memory, on their way until the thread waits for its cp.async group.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// The batch as gemm_serving.h describes it. Sizes are checked on the host so that every
// combined key index (prefix + own) fits an int.
struct BatchView {
    const int *q_start, *kv_lens, *table;
    int64_t table_stride;
    int num_seqs, num_tokens, table_width;
    int num_pages, page_shift;   // of the cache
    int prefix_len;              // keys, whole pages
};

// One sequence, limited to what may be accessed: tokens [q0, q0 + n), kv own keys. `bad`: a
// value had to be limited.
struct SeqView {
    int q0, n, kv;
    bool bad;
};

// A value of q_start. No operator writes it, so it may be read as data that no one writes while the kernel runs; kv_lens may come from
// the kernel before (see grid_dependency_wait). With ordinary loads attention of drafts over heads of 64 took 94.4 us for 79.5.
__host__ __device__ __forceinline__ int load_start(const int *at)
{
#ifdef __CUDA_ARCH__
    return __ldg(at);
#else
    return *at;
#endif
}

__host__ __device__ __forceinline__ SeqView load_seq(const BatchView &b, int s)
{
    const int q0 = load_start(b.q_start + s), q1 = load_start(b.q_start + s + 1), kv = b.kv_lens[s];
    const int cap = b.table_width << b.page_shift;
    SeqView v;
    v.q0 = min(max(q0, 0), b.num_tokens);
    const int end = min(max(q1, v.q0), b.num_tokens);
    v.n = end - v.q0;
    v.kv = min(max(kv, 0), cap);
    v.bad = v.q0 != q0 || end != q1 || v.kv != kv;
    return v;
}

// Sequence of `token`: the largest s with q_start[s] <= token, found by the L lanes of a group
// together (L + 1 parts per step). All lanes of the warp take part.
template <int L>
__device__ __forceinline__ int find_seq(const int *q_start, int num_seqs, int token, int lane)
{
    const int sub = lane % L, first = lane - sub;
    int lo = 0;
    for (int width = num_seqs; width > 1;) {
        const int step = (width + L - 1) / L;
        const int at = lo + (sub + 1) * step;
        const bool below = at < num_seqs && load_start(q_start + at) <= token;
        const uint32_t votes = (__ballot_sync(0xffffffffu, below) >> first) & (0xffffffffu >> (32 - L));
        lo += __popc(votes) * step;
        width = step;
    }
    return min(lo, num_seqs - 1);   // a table that is not sorted may lead past the end
}

}  // namespace gb300
