// Norm and rotation of query and key heads, with the outputs in strided tensors (gemm_qk_rope)
// or the keys and values in a paged cache (gemm_kv_append).
//
//     y = x / sqrt(mean(x^2) + eps) * w                       (per head, if there are weights)
//     (a, b) -> scale * (a cos t - b sin t, b cos t + a sin t)  t = 2 pi * frac(p * f)
//
// over pairs of the first rotary_dim values. The turns f of a pair per position are held in
// units of 2^-64, so that p * f modulo one turn is one wrapping 64-bit product, exact at any
// position: the angle's error is that of the table's rounding, p * 2^-65 turns, where an FP32
// product is off by 0.06 rad at a million positions and an FP64 one costs the FP64 units (a few
// operations per clock and SM).
//
// Bound by memory: every value is read once and written once. A group of head_dim / 8 lanes
// takes one token and `heads_per_item` of its heads, 16 bytes per lane and head, four heads in
// flight; a lane's dimensions are the same for all of them, so cosines and sines are computed
// once per group, the pair partner (half layout) and the sum of squares go through shuffles, and
// nothing needs shared memory or a barrier.
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
    HeadsView q, k, v;            // in the order of a token's heads; v is copied
    int tokens, chunks, heads_per_item;
    const int *positions;         // not paged
    BatchView batch;              // paged
    int64_t row_stride;           // paged: of the cache
    const uint64_t *table;
    const void *q_norm, *k_norm;
    int rotary_dim, interleaved;
    float eps, scale;
    uint32_t *err;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeInFlight = 4;   // heads loaded before the first is worked on

template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p)
{
    constexpr int L = D / 8;   // lanes per token
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, sub = lane % L;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / L) + threadIdx.x / L;
    const int64_t token64 = item / p.chunks;
    const int chunk = static_cast<int>(item - token64 * p.chunks);
    bool live = token64 < p.tokens;
    const int token = live ? static_cast<int>(token64) : p.tokens - 1;

    // the token's position, and its row of the cache
    int64_t pos, cache_row = -1;
    if constexpr (PAGED) {
        const int s = find_seq<L>(p.batch.q_start, p.batch.num_seqs, token, lane);
        const SeqView seq = load_seq(p.batch, s);
        live = live && token >= seq.q0 && token < seq.q0 + seq.n;
        const int64_t place = static_cast<int64_t>(seq.kv) - seq.n + (token - seq.q0);
        pos = p.batch.prefix_len + place;
        bool bad = seq.bad;
        if (live && place >= 0) {   // place < kv <= the keys of table_width pages
            const int page = __ldg(p.batch.table + s * p.batch.table_stride + (place >> p.batch.page_shift));
            if (page >= 0 && page < p.batch.num_pages)
                cache_row = (static_cast<int64_t>(page) << p.batch.page_shift) + (place & ((1 << p.batch.page_shift) - 1));
        }
        bad = bad || (live && cache_row < 0);
        if (bad && sub == 0)
            atomicCAS(p.err, 0u, static_cast<uint32_t>(ERR_BATCH_INDEX));
    } else {
        pos = __ldg(p.positions + token);
    }

    // cosine and signed sine of this lane's eight values: y[e] = x[e] * cs[e] + partner[e] * sn[e]
    const int d0 = sub * 8, half = p.rotary_dim / 2;
    const bool rotates = d0 < p.rotary_dim;
    const bool second = !p.interleaved && d0 >= half;
    float cs[8] = {}, sn[8] = {};
    auto angle = [&](int pair, float &c, float &s) {
        const uint64_t turns = static_cast<uint64_t>(pos) * __ldg(p.table + pair);
        // the top 32 bits as a signed part of a turn, in half turns (2^-31 each)
        const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
        sincospif(x, &s, &c);
        c *= p.scale;
        s *= p.scale;
    };
    if (rotates && p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            angle(d0 / 2 + e, cs[2 * e], sn[2 * e + 1]);
            cs[2 * e + 1] = cs[2 * e];
            sn[2 * e] = -sn[2 * e + 1];
        }
    } else if (rotates) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            angle(d0 - (second ? half : 0) + e, cs[e], sn[e]);
            sn[e] = second ? sn[e] : -sn[e];
        }
    }
    const int partner = rotates && !p.interleaved ? lane + (second ? -half / 8 : half / 8) : lane;

    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if (p.q_norm)
        wq = __ldg(static_cast<const uint4 *>(p.q_norm) + sub);
    if (p.k_norm)
        wk = __ldg(static_cast<const uint4 *>(p.k_norm) + sub);

    const int all = p.q.heads + p.k.heads + p.v.heads;
    const int h_end = min(all, (chunk + 1) * p.heads_per_item);
    // (every lane runs the same number of steps: the shuffles below are warp-wide)
    for (int i0 = 0; i0 < p.heads_per_item; i0 += kRopeInFlight) {
        uint4 x[kRopeInFlight];
        T *dst[kRopeInFlight];
        int kind[kRopeInFlight];   // 0 query, 1 key, 2 value
#pragma unroll
        for (int u = 0; u < kRopeInFlight; ++u) {
            const int h = chunk * p.heads_per_item + i0 + u;
            const bool on = live && i0 + u < p.heads_per_item && h < h_end;
            kind[u] = h < p.q.heads ? 0 : h < p.q.heads + p.k.heads ? 1 : 2;
            const HeadsView &g = kind[u] == 0 ? p.q : kind[u] == 1 ? p.k : p.v;
            const int hh = kind[u] == 0 ? h : kind[u] == 1 ? h - p.q.heads : h - p.q.heads - p.k.heads;
            dst[u] = nullptr;
            x[u] = make_uint4(0, 0, 0, 0);
            if (on) {
                x[u] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(g.in) + token * g.in_token + hh * g.in_head + d0);
                if (!PAGED || kind[u] == 0)
                    dst[u] = static_cast<T *>(g.out) + token * g.out_token + hh * g.out_head + d0;
                else if (cache_row >= 0)
                    dst[u] = static_cast<T *>(g.out) + (cache_row >> p.batch.page_shift) * g.out_token + hh * g.out_head +
                             (cache_row & ((1 << p.batch.page_shift) - 1)) * p.row_stride + d0;
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeInFlight; ++u) {
            float f[8];
            const uint32_t raw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = unpack2<T>(raw[e]);
                f[2 * e] = v.x;
                f[2 * e + 1] = v.y;
            }
            if (p.q_norm || p.k_norm) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss = fmaf(f[e], f[e], ss);
#pragma unroll
                for (int o = L / 2; o > 0; o /= 2)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const uint4 w = kind[u] == 0 ? wq : wk;
                if (kind[u] == 0 ? p.q_norm != nullptr : kind[u] == 1 && p.k_norm) {
                    const float r = rsqrtf(ss * (1.0f / D) + p.eps);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = unpack2<T>(ww[e]);
                        f[2 * e] = f[2 * e] * r * v.x;
                        f[2 * e + 1] = f[2 * e + 1] * r * v.y;
                    }
                }
            }
            float y[8];
            if (p.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = fmaf(f[e], cs[e], f[e ^ 1] * sn[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = fmaf(f[e], cs[e], __shfl_sync(0xffffffffu, f[e], partner) * sn[e]);
            }
            uint4 r;
            r.x = rotates ? pack2<T>(y[0], y[1]) : pack2<T>(f[0], f[1]);
            r.y = rotates ? pack2<T>(y[2], y[3]) : pack2<T>(f[2], f[3]);
            r.z = rotates ? pack2<T>(y[4], y[5]) : pack2<T>(f[4], f[5]);
            r.w = rotates ? pack2<T>(y[6], y[7]) : pack2<T>(f[6], f[7]);
            if (kind[u] == 2)
                r = x[u];   // bit for bit, NaN payloads too
            if (dst[u])
                *reinterpret_cast<uint4 *>(dst[u]) = r;
        }
    }
}

}  // namespace gb300
