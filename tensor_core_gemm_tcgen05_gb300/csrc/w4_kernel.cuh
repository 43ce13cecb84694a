// C[M][N] = act(A[M][K] W^T + bias[N]) with W[n][k] = (code - zero) scale, 4-bit codes (gemm_decode.h), for few rows
// of A: what the time goes to is reading W once.
//
// The rows of W are the rows of 16 x 8 x 16 products and come straight into registers, the rows of A (tokens) are
// the columns. Codes become code - zero exactly: the four bits go into the mantissa of 1024 (FP16) or 128 (BF16), from
// which 1024 + zero or 128 + zero is taken. Each group is summed by itself in FP32 and its sum scaled in FP32, so that
// no weight is rounded.
//
// A warp takes 16 rows of W in steps of 128 columns; ROWS_W warps of a CTA stand side by side, the others
// and (in a cluster) other CTAs share the columns; the partial sums meet in shared and distributed shared memory in a
// fixed order. A is brought to shared memory a chunk of steps at a time, in the order the products take it.
#pragma once

#include "mma_sync.cuh"
#include "serving_common.cuh"

namespace gb300 {

constexpr int kW4Threads = 256, kW4Warps = 8;
constexpr int kW4Ahead = 4;   // steps whose codes a warp has in flight

struct W4Params {
    int M, N, K;
    const void *a;
    int64_t lda;
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros;   // or nullptr: 8
    const void *bias;       // or nullptr
    void *c;
    int64_t ldc;
    int epilogue;
    int row_warps;   // of a CTA: 1, 2, 4 or 8
    int steps;       // of 128 columns, the last maybe in part
};

// The activation in FP32 (NaN stays NaN).
__device__ __forceinline__ void w4_activate(int epilogue, float &x0, float &x1)
{
    if (epilogue == EPI_GELU) {
        float y0 = x0, y1 = x1;
        gelu_pair(y0, y1);
        x0 = fabsf(x0) < 16.0f ? y0 : x0 < 0.0f ? -0.0f : x0;   // (beyond: x or nothing, to FP32's last bit)
        x1 = fabsf(x1) < 16.0f ? y1 : x1 < 0.0f ? -0.0f : x1;
    } else if (epilogue == EPI_RELU) {
        x0 = x0 < 0.0f ? 0.0f : x0;
        x1 = x1 < 0.0f ? 0.0f : x1;
    }
}

// Codes j and j + 4 of a word of eight (the first in the lowest bits), minus zero, as pair j of x. The constants of a
// zero: what is to be taken from the pairs.
template <typename T>
struct W4Codes;
template <>
struct W4Codes<__half> {
    __half2 z, z16;
    __device__ __forceinline__ explicit W4Codes(uint32_t zero)
    {
        const uint32_t one = 0x6400u | zero, sixteenth = 0xd400u | zero << 4;   // 1024 + zero, -(64 + zero)
        const uint32_t a = one * 0x10001u, b = sixteenth * 0x10001u;
        z = *reinterpret_cast<const __half2 *>(&a);
        z16 = *reinterpret_cast<const __half2 *>(&b);
    }
    __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&x)[4]) const
    {
        const uint32_t one16 = 0x2c002c00u;   // 1 / 16
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = (w & 0x000f000fu) | 0x64006400u;   // 1024 + code
            const uint32_t hi = (w & 0x00f000f0u) | 0x64006400u;   // 1024 + 16 code
            const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), z);
            const __half2 b = __hfma2(*reinterpret_cast<const __half2 *>(&hi), *reinterpret_cast<const __half2 *>(&one16), z16);
            x[2 * h] = *reinterpret_cast<const uint32_t *>(&a);
            x[2 * h + 1] = *reinterpret_cast<const uint32_t *>(&b);
            w >>= 8;
        }
    }
};
template <>
struct W4Codes<__nv_bfloat16> {
    __nv_bfloat162 z;
    __device__ __forceinline__ explicit W4Codes(uint32_t zero)
    {
        const uint32_t a = (0x4300u | zero) * 0x10001u;   // 128 + zero
        z = *reinterpret_cast<const __nv_bfloat162 *>(&a);
    }
    __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&x)[4]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = (w & 0x000f000fu) | 0x43004300u;
            const __nv_bfloat162 a = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), z);
            x[j] = *reinterpret_cast<const uint32_t *>(&a);
            w >>= 4;
        }
    }
};

// A step's codes of a lane: 32 of row g and 32 of row g + 8, and (lane t, t < groups of the step) scale and
// zero of group t in both rows.
struct W4Step {
    uint32_t w[2][4];
    uint32_t sz[2];   // scale's bits, zero << 16
};

template <typename T>
__device__ __forceinline__ float w4_scale(uint32_t sz)
{
    return unpack2<T>(sz & 0xffffu).x;
}

// GW: words of eight codes that a lane has of a group (1, 2, 4: groups of 32, 64, 128). TILES: of eight rows of A.
template <typename T, int TILES, int GW>
__global__ void __launch_bounds__(kW4Threads) w4_kernel(const __grid_constant__ W4Params p)
{
    constexpr int GROUPS = 4 / GW, GROUP = 32 * GW;   // groups of a step
    extern __shared__ uint4 act[];                    // [step of the chunk][word][tile][lane]
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint32_t ctas, rank = cluster_ctarank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int row_warp = warp % p.row_warps, k_warp = warp / p.row_warps, k_warps = kW4Warps / p.row_warps;
    const int rows = 16 * p.row_warps;   // of W in this CTA
    const int n0 = static_cast<int>(blockIdx.x / ctas) * rows, m0 = static_cast<int>(blockIdx.y) * TILES * 8;
    const int step0 = static_cast<int>(static_cast<int64_t>(p.steps) * rank / ctas);
    const int step1 = static_cast<int>(static_cast<int64_t>(p.steps) * (rank + 1) / ctas);
    const int chunk = kW4Ahead * k_warps;   // steps
    const int groups = p.K / GROUP;
    // ---- codes
    int64_t row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        row[h] = min(n0 + 16 * row_warp + 8 * h + g, p.N - 1);   // (rows past the last are not written)
    auto load = [&](int step, W4Step &x) {
        const bool on = step < step1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *src = p.codes + row[h] * (p.K / 2) + static_cast<int64_t>(step) * 64;
            if constexpr (GW == 4) {
                const uint4 v = on ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * t)) : make_uint4(0, 0, 0, 0);
                x.w[h][0] = v.x, x.w[h][1] = v.y, x.w[h][2] = v.z, x.w[h][3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < GROUPS; ++i) {
                    const bool in = on && step * GROUPS + i < groups;
                    if constexpr (GW == 2) {
                        const uint2 v = in ? __ldg(reinterpret_cast<const uint2 *>(src + 32 * i + 8 * t)) : make_uint2(0, 0);
                        x.w[h][2 * i] = v.x, x.w[h][2 * i + 1] = v.y;
                    } else {
                        x.w[h][i] = in ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * i + 4 * t)) : 0u;
                    }
                }
            }
            uint32_t sz = 8u << 16;   // past the last group: scale 0
            if (on && t < GROUPS && step * GROUPS + t < groups) {
                const int64_t at = row[h] * groups + step * GROUPS + t;
                const uint32_t zero = p.zeros ? __ldg(p.zeros + at) & 15u : 8u;
                sz = __ldg(static_cast<const uint16_t *>(p.scales) + at) | zero << 16;
            }
            x.sz[h] = sz;
        }
    };
    float acc[TILES][4] = {};
    W4Step x[kW4Ahead];
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u)
        load(step0 + u * k_warps + k_warp, x[u]);
    for (int first = step0; first < step1; first += chunk) {
        // ---- A's columns of this chunk
        if (first > step0)
            __syncthreads();
        const int steps = min(chunk, step1 - first);
        for (int i = threadIdx.x; i < TILES * 8 * steps * 16; i += kW4Threads) {
            const int k8 = i % (steps * 16), m = i / (steps * 16), at = k8 % 16;
            const int64_t k = static_cast<int64_t>(first) * 128 + 8 * k8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (m0 + m < p.M && k < p.K)
                v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.a) + (m0 + m) * p.lda + k));
            // eight columns belong to one lane's word; the word's pairs are columns j and j + 4
            const int lane_t = GW == 4 ? at / 4 : GW == 2 ? at / 2 % 4 : at % 4;
            const int word = GW == 4 ? at % 4 : GW == 2 ? at / 8 * 2 + at % 2 : at / 4;
            act[((k8 / 16 * 4 + word) * TILES + m / 8) * 32 + m % 8 * 4 + lane_t] =
                make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
        }
        __syncthreads();
        // ---- products
#pragma unroll
        for (int u = 0; u < kW4Ahead; ++u) {
            const int at = u * k_warps + k_warp;   // step of the chunk
            if (at < steps) {
#pragma unroll
                for (int i = 0; i < GROUPS; ++i) {
                    const uint32_t sz0 = __shfl_sync(0xffffffffu, x[u].sz[0], (lane & ~3) | i);
                    const uint32_t sz1 = __shfl_sync(0xffffffffu, x[u].sz[1], (lane & ~3) | i);
                    const W4Codes<T> z0(sz0 >> 16), z1(sz1 >> 16);
                    float sum[TILES][4] = {};
#pragma unroll
                    for (int w = i * GW; w < (i + 1) * GW; ++w) {
                        uint32_t a0[4], a1[4];
                        z0.unpack(x[u].w[0][w], a0);
                        z1.unpack(x[u].w[1][w], a1);
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            const uint4 b = act[((at * 4 + w) * TILES + n) * 32 + lane];
                            mma_16x8x16<T>(sum[n], a0[0], a1[0], a0[1], a1[1], b.x, b.y);
                            mma_16x8x16<T>(sum[n], a0[2], a1[2], a0[3], a1[3], b.z, b.w);
                        }
                    }
                    const float s0 = w4_scale<T>(sz0), s1 = w4_scale<T>(sz1);
#pragma unroll
                    for (int n = 0; n < TILES; ++n) {
                        acc[n][0] = fmaf(sum[n][0], s0, acc[n][0]);
                        acc[n][1] = fmaf(sum[n][1], s0, acc[n][1]);
                        acc[n][2] = fmaf(sum[n][2], s1, acc[n][2]);
                        acc[n][3] = fmaf(sum[n][3], s1, acc[n][3]);
                    }
                }
            }
            load(first + chunk + at, x[u]);
        }
    }
    // ---- partial sums: [k warp][token][row of W], tokens 4 words further apart than a row is long
    const int pitch = rows + 4;
    float *part = reinterpret_cast<float *>(act);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < TILES; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            part[(k_warp * TILES * 8 + 8 * n + 2 * t + e % 2) * pitch + 16 * row_warp + g + e / 2 * 8] = acc[n][e];
    __syncthreads();
    if (k_warps > 1) {
        for (int i = threadIdx.x; i < TILES * 8 * rows; i += kW4Threads) {
            const int at = i / rows * pitch + i % rows;
            float sum = part[at];
            for (int w = 1; w < k_warps; ++w)
                sum += part[w * TILES * 8 * pitch + at];
            part[at] = sum;
        }
        __syncthreads();
    }
    if (ctas > 1)
        cluster_sync();
    // this CTA's share of the outputs: pairs of rows of W for one token
    const int pairs = TILES * 8 * rows / 2, share = (pairs + static_cast<int>(ctas) - 1) / static_cast<int>(ctas);
    const uint32_t base = smem_u32(part);
    for (int i = static_cast<int>(rank) * share + static_cast<int>(threadIdx.x); i < min(pairs, (static_cast<int>(rank) + 1) * share);
         i += kW4Threads) {
        const int m = i / (rows / 2), r = i % (rows / 2) * 2;
        if (m0 + m >= p.M || n0 + r >= p.N)
            continue;
        float2 y = make_float2(0.0f, 0.0f);
        if (ctas == 1) {   // (shared::cluster addresses only come from mapa, in a cluster)
            y = *reinterpret_cast<const float2 *>(part + m * pitch + r);
        } else {
            for (uint32_t c = 0; c < ctas; ++c) {
                const float2 v = ld_shared_cluster_f2(mapa_shared(base + static_cast<uint32_t>(m * pitch + r) * 4u, c));
                y.x += v.x;
                y.y += v.y;
            }
        }
        if (p.bias) {
            const float2 b = unpack2<T>(__ldg(reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.bias) + n0 + r)));
            y.x += b.x;
            y.y += b.y;
        }
        w4_activate(p.epilogue, y.x, y.y);
        *reinterpret_cast<uint32_t *>(static_cast<T *>(p.c) + (m0 + m) * p.ldc + n0 + r) = pack2<T>(y.x, y.y);
    }
    __syncthreads();
    if (ctas > 1)
        cluster_sync();   // the other CTAs have read this one's sums
}

}  // namespace gb300
