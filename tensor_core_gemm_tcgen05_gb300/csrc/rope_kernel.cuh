// Norm and rotation of query and key heads, with the outputs in strided tensors (gemm_qk_rope)
// or the keys and values in a paged cache (gemm_kv_append).
//
//     y = x / sqrt(mean(x^2) + eps) * w                       (per head, if there are weights)
//     (a, b) -> scale * (a cos t - b sin t, b cos t + a sin t)  t = 2 pi * frac(p * f)
//
// over pairs of the first rotary_dim values. The turns f of a pair per position are held in
// units of 2^-64, so that p * f modulo one turn is one wrapping 64-bit product, which adds no error
// at any position. The angle's error is p times the table's (gemm_rope_table computes in FP64: up to 2^-55 turns for
// the fastest pairs) and 2^-26 of a turn everywhere, from the float in which the fraction's top 32 bits go to the sine.
// An FP32 product is off by 0.06 rad at a million positions, and an FP64 one costs the FP64 units (a few
// operations per clock and SM).
//
// Bound by memory: every value is read once and written once. A group of head_dim / 8 lanes
// takes one token and up to `heads_per_item` of its query, its key or its value heads, 16 bytes
// per lane and head, kRopeInFlight heads in flight. A lane's dimensions are the same for all of
// them, so its cosines and sines, times the norm's weights, are computed once per group (in the
// half layout the two lanes of a pair compute half of them each); the pair's other value and the
// sum of squares go through shuffles, and nothing needs shared memory or a barrier. The first
// heads are loaded before the token's sequence is looked up.
#pragma once

#include "serving_common.cuh"

namespace gb300 {

struct HeadsView {
    const void *in;
    int64_t in_token, in_head;     // strides in elements
    void *out;
    int64_t out_token, out_head;   // paged keys and values: out_token is the page stride
    int heads;
};

struct RopeParams {
    HeadsView q, k, v;                // v is copied
    int tokens, heads_per_item;
    int q_chunks, k_chunks, chunks;   // items of a token: its query heads', key heads', all
    const int *positions;             // not paged
    BatchView batch;                  // paged
    int64_t row_stride;               // paged: of the cache
    const uint64_t *table;
    const void *q_norm, *k_norm;
    int rotary_dim, interleaved;
    float eps, scale;
    uint32_t *err;
};

// 64 registers a thread: 1024 threads per SM, 64 KB of heads in flight (8200 tokens, 32 + 32 heads of
// 128: 42.8 us, 6.28 TB/s; 256-thread blocks 43.6; five of those per SM, spilling, 81; three 46.5;
// two heads in flight 76, eight 46.9). Streaming stores or loads: 3 % slower.
constexpr int kRopeThreads = 128;
constexpr int kRopeInFlight = 4;   // heads loaded before the first is worked on

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8])
{
    const uint32_t raw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = unpack2<T>(raw[e]);
        f[2 * e] = v.x;
        f[2 * e + 1] = v.y;
    }
}

template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int L = D / 8;   // lanes per token
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, sub = lane % L, d0 = sub * 8;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / L) + threadIdx.x / L;
    const int64_t token64 = item / p.chunks;
    int chunk = static_cast<int>(item - token64 * p.chunks);
    const bool in_range = token64 < p.tokens;
    const int token = in_range ? static_cast<int>(token64) : p.tokens - 1;
    const int kind = chunk < p.q_chunks ? 0 : chunk < p.q_chunks + p.k_chunks ? 1 : 2;   // query, key, value
    chunk -= kind == 0 ? 0 : kind == 1 ? p.q_chunks : p.q_chunks + p.k_chunks;
    const HeadsView &g = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const int h0 = chunk * p.heads_per_item, h1 = min(g.heads, h0 + p.heads_per_item);

    uint4 x[kRopeInFlight];
    const T *src = static_cast<const T *>(g.in) + token * g.in_token + h0 * g.in_head + d0;
    const int64_t in_head = g.in_head;
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kRopeInFlight; ++u) {
            x[u] = make_uint4(0, 0, 0, 0);
            if (in_range && h0 + i0 + u < h1)
                x[u] = *reinterpret_cast<const uint4 *>(src + (i0 + u) * in_head);
        }
    };
    load(0);

    // the token's position, and where its heads go
    int64_t pos;
    bool live = in_range;
    T *dst = static_cast<T *>(g.out) + token * g.out_token;
    if constexpr (PAGED) {
        const int s = find_seq<L>(p.batch.q_start, p.batch.num_seqs, token, lane);
        const SeqView seq = load_seq(p.batch, s);
        live = live && token >= seq.q0 && token < seq.q0 + seq.n;
        const int64_t place = static_cast<int64_t>(seq.kv) - seq.n + (token - seq.q0);
        pos = p.batch.prefix_len + place;
        bool bad = seq.bad;
        if (kind != 0 && live) {
            int page = -1;
            if (place >= 0)   // place < kv <= the keys of table_width pages
                page = p.batch.table[s * p.batch.table_stride + (place >> p.batch.page_shift)];
            live = page >= 0 && page < p.batch.num_pages;
            bad = bad || !live;
            dst = static_cast<T *>(g.out) + page * g.out_token + (place & ((1 << p.batch.page_shift) - 1)) * p.row_stride;
        }
        // the threads of the grid look at all sequences, those without tokens here too
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x; i < p.batch.num_seqs;
             i += static_cast<int64_t>(gridDim.x) * kRopeThreads)
            bad = bad || load_seq(p.batch, static_cast<int>(i)).bad;
        if (bad)
            atomicCAS(p.err, 0u, static_cast<uint32_t>(ERR_BATCH_INDEX));
    } else {
        pos = p.positions[token];
    }
    dst += h0 * g.out_head + d0;
    const int64_t out_head = g.out_head;

    // y[e] = x[e] * cs[e] + partner[e] * sn[e], with the norm's weights in the factors
    const int half = p.rotary_dim / 2;
    const bool rotates = d0 < p.rotary_dim && kind != 2, pairs = d0 < p.rotary_dim && !p.interleaved;
    const bool second = pairs && d0 >= half;
    const int partner = pairs ? lane + (second ? -half / 8 : half / 8) : lane;
    float cs[8], sn[8];
    {
        float c4[4], s4[4];   // of four pairs
        const int pair0 = p.interleaved ? d0 / 2 : d0 - (second ? half - 4 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c4[e] = 1.0f;
            s4[e] = 0.0f;
            if (d0 < p.rotary_dim) {
                const uint64_t turns = static_cast<uint64_t>(pos) * p.table[pair0 + e];
                // the top 32 bits as a signed part of a turn, in half turns (2^-31 each)
                sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f, &s4[e], &c4[e]);
                c4[e] *= p.scale;
                s4[e] *= p.scale;
            }
        }
        if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[2 * e] = cs[2 * e + 1] = c4[e];
                sn[2 * e] = -s4[e];
                sn[2 * e + 1] = s4[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float co = __shfl_sync(0xffffffffu, c4[e], partner), so = __shfl_sync(0xffffffffu, s4[e], partner);
                cs[e] = second ? co : c4[e];
                cs[e + 4] = second ? c4[e] : co;
                sn[e] = second ? so : -s4[e];
                sn[e + 4] = second ? s4[e] : -so;
            }
        }
    }
    const void *norm = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
    if (norm) {
        float w[8], wp[8];
        unpack8<T>(static_cast<const uint4 *>(norm)[sub], w);
        unpack8<T>(static_cast<const uint4 *>(norm)[partner % L], wp);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cs[e] *= w[e];
            sn[e] *= p.interleaved ? w[e ^ 1] : wp[e];
        }
    }

    // (every lane runs the same number of steps: the shuffles are warp-wide)
    const bool any_norm = p.q_norm || p.k_norm;
    for (int i0 = 0;;) {
#pragma unroll
        for (int u = 0; u < kRopeInFlight; ++u) {
            float f[8], y[8];
            unpack8<T>(x[u], f);
            float r = 1.0f;
            if (any_norm) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss = fmaf(f[e], f[e], ss);
#pragma unroll
                for (int o = L / 2; o > 0; o /= 2)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = norm ? rsqrtf(ss * (1.0f / D) + p.eps) : 1.0f;
            }
            if (p.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = f[e] * cs[e];
                    if (rotates)
                        y[e] = fmaf(f[e ^ 1], sn[e], y[e]);
                }
            } else {
                uint4 xp;
                xp.x = __shfl_sync(0xffffffffu, x[u].x, partner);
                xp.y = __shfl_sync(0xffffffffu, x[u].y, partner);
                xp.z = __shfl_sync(0xffffffffu, x[u].z, partner);
                xp.w = __shfl_sync(0xffffffffu, x[u].w, partner);
                float fp[8];
                unpack8<T>(xp, fp);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = f[e] * cs[e];
                    if (rotates)
                        y[e] = fmaf(fp[e], sn[e], y[e]);
                }
            }
            uint4 out = x[u];   // values: bit for bit, NaN payloads too
            if (kind != 2)
                out = make_uint4(pack2<T>(y[0] * r, y[1] * r), pack2<T>(y[2] * r, y[3] * r), pack2<T>(y[4] * r, y[5] * r),
                                 pack2<T>(y[6] * r, y[7] * r));
            if (live && h0 + i0 + u < h1)
                *reinterpret_cast<uint4 *>(dst + (i0 + u) * out_head) = out;
        }
        i0 += kRopeInFlight;
        if (i0 >= p.heads_per_item)
            break;
        load(i0);
    }
}

}  // namespace gb300
