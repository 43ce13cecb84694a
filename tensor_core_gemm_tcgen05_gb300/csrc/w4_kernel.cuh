// C[M][N] = act(A[M][K] W^T + bias[N]) with W[n][k] = (code - zero) scale, 4-bit codes (gemm_decode.h), for up to eight
// rows of A: what the time goes to is reading W once. (w4_umma_kernel.cuh has the form for more rows.)
//
// The rows of W are the rows of 16 x 8 x 16 products and come straight into registers, the rows of A (tokens) are
// the columns. With the zero z, the scale s and the columns of a group,
//     s sum (code - z) x = s (sum code x - z sum x),
// so the products are of the codes themselves, which cost a mask each (see W4Codes) and are exact, and sum x comes with A. Groups
// are summed and scaled in FP32: no weight is rounded. Where x is so large that code x or z sum x may leave FP32's range (BF16 from
// 2^113 on, infinities, NaN) the two terms would cancel to NaN: a CTA that finds such a value takes code - zero itself to the products.
//
// A stays: a CTA (one to an SM, sixteen warps) brings its columns of A to shared memory once, in the order the products take
// them, and then sees the tiles of 16 rows of W that are its cluster's, eight, four, two or one at a time (a round), the columns
// of a tile shared by the other warps and by the CTAs of the cluster (several, where A does not fit one). A step is 256 columns
// of a tile; each lane copies its own codes of the next steps into a ring of its own, across rounds, so nothing but the
// sums of a round waits for another warp. These meet in shared and distributed shared memory in a fixed order.
//
// What bounds it: the chain of a step in its sixteen warps (issue 1.6 a cycle and SM, of which unpacking is a third; HBM at 24 %)
// behind a start of about 3 us. Measured (captured, weights from HBM): 4096 x 4096 6.1 us for one row, 7.0 for eight, 16384 x 4096
// 14.3 and 15.4 (33.5 MB: 5.2 at the copy rate), 32768 x 4096 20.7 and 21.7, 1024 x 1024 3.7 and 3.8. What it took there before:
// steps of 128 columns with a ring of four 25 (eight rows, 16384 x 4096); codes - zero unpacked for each row 24; 256 threads that
// brought A anew for each 128 rows 23; two more barriers to a round 17.2.
//
// Laying A out is 1 of the 14.3 and about 2.5 of the 15.4. While the eight rows took 15.8: four pieces in flight whatever their number 14.6 and
// 16.5; eight 15.0 and 15.6; sums always as products with ones, which need a barrier and a look at all groups, 14.6 and 15.1 (4096 x
// 4096, one row 6.5 for 6.1); asynchronous copies to the pieces' places, then a turn in place, 15.4 and 18.6.
#pragma once

#include <type_traits>

#include "mma_sync.cuh"
#include "serving_common.cuh"

namespace gb300 {

constexpr int kW4Threads = 512, kW4LogWarps = 4, kW4Warps = 1 << kW4LogWarps;
constexpr int kW4Round = 8;   // tiles of 16 rows of W in a round, at most (4: 32768 x 4096, one row 22.1 us for 21.0)
constexpr int kW4Rows = 8;    // of A in a CTA
constexpr int kW4Ahead = 2;   // steps whose codes a warp has in flight

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
    int tiles, clusters;   // w4_kernel: of 16 rows of W; of CTAs
    int slice;             // w4_kernel: steps of a CTA, at most
    int steps;             // of 256 (w4_kernel) or 128 columns, the last maybe in part
    uint32_t *err;
    uint64_t timeout_ns;
    int debug;             // DEBUG_WITHHOLD_FIRST_LOAD (w4_umma_kernel)
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

// Codes j and j + 4 of a word of eight (the first in the lowest bits) as pair j of x, so that the value of a pair's bits
// times UNIT (j even) or ODD_UNIT (j odd) is BASE + code.
//  * FP16: bits alone are subnormal numbers, code 2^-24; odd codes are left where they are, 16 code 2^-24.
//  * BF16: in the mantissa of 128. (As subnormal numbers times x they would leave FP32's range.) The sums then lose
//    5 of FP32's 24 bits to the base, of which the result keeps 8.
// A group's sums, and what is taken off them, stay in FP32's range where all |x| are below LIMIT: FP16 128 15 2^16, BF16 128 143 2^113 < 2^128.
template <typename T>
struct W4Codes;
template <>
struct W4Codes<__half> {
    static constexpr float UNIT = 16777216.0f, ODD_UNIT = 1048576.0f, BASE = 0.0f;
    static constexpr uint32_t ONES = 0x3c003c00u;   // two of them
    static constexpr float LIMIT = INFINITY;
    static __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&x)[4])
    {
        x[0] = w & 0x000f000fu;
        x[1] = w & 0x00f000f0u;
        w >>= 8;
        x[2] = w & 0x000f000fu;
        x[3] = w & 0x00f000f0u;
    }
};
template <>
struct W4Codes<__nv_bfloat16> {
    static constexpr float UNIT = 1.0f, ODD_UNIT = 1.0f, BASE = 128.0f;
    static constexpr uint32_t ONES = 0x3f803f80u;
    static constexpr float LIMIT = 1.0384593717069655e34f;   // 2^113
    static __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&x)[4])
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
    }
};

// The same with code - zero (BF16: times 2^-11, so that a group's sum stays in FP32's range whatever the 128 values are) as the value, a
// zero for each row. Times MINUS_ZERO_UNIT it is the value itself.
template <typename T>
constexpr float MINUS_ZERO_UNIT = std::is_same<T, __half>::value ? 1.0f : 2048.0f;
template <typename T>
__device__ __forceinline__ void w4_unpack_minus_zero(uint32_t w, uint32_t zero, uint32_t (&x)[4])
{
    constexpr bool HALF = std::is_same<T, __half>::value;
    const uint32_t base = HALF ? 0x64006400u : 0x43004300u;   // 1024 or 128
    const uint32_t less = (HALF ? base : 0xbd80bd80u) | zero * 0x10001u, times = 0x3a003a00u;   // with the zero; BF16: times -2^-11; 2^-11
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | base;
        if constexpr (HALF) {
            const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&less));
            x[j] = *reinterpret_cast<const uint32_t *>(&y);
        } else {
            const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&times),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&less));
            x[j] = *reinterpret_cast<const uint32_t *>(&y);
        }
    }
}

// A warp's way through the rounds of its cluster's tiles: 2^log_rows tiles from `tile` on; of a tile its steps w, w + warps, ...,
// in `turns` turns, a multiple of kW4Ahead (so that a turn's slot of the ring is known when compiling; the last may be empty).
struct W4Walk {
    int tile, left, log_rows, step, turns;
    __device__ __forceinline__ void begin(int warp, int count)
    {
        static_assert(kW4Round == 8 && kW4Ahead == 2, "powers of two below");
        log_rows = left >= 8 ? 3 : left >= 4 ? 2 : left >= 2 ? 1 : 0;
        step = warp >> log_rows;
        turns = ((count + (2 * kW4Warps >> log_rows) - 1) >> (kW4LogWarps + 1 - log_rows)) * kW4Ahead;
    }
    __device__ __forceinline__ void end_round(int warp, int count)
    {
        tile += 1 << log_rows;
        left -= 1 << log_rows;
        begin(warp, count);
    }
    __device__ __forceinline__ int row_warp(int warp) const { return warp & ((1 << log_rows) - 1); }
    __device__ __forceinline__ int warps() const { return kW4Warps >> log_rows; }   // of a tile
};

// A warp's pieces of 256 columns of A's rows, `count` to a row: the warp-th of all and every kW4Warps-th from there on. (No division:
// it would cost as much as the rest.)
struct W4Pieces {
    int row = 0, piece;
    __device__ __forceinline__ W4Pieces(int warp, int count) : piece(warp) { settle(count); }
    __device__ __forceinline__ void next(int count)
    {
        piece += kW4Warps;
        settle(count);
    }
    __device__ __forceinline__ void settle(int count)
    {
        for (; piece >= count && row < kW4Rows; ++row)
            piece -= count;
    }
};

// Bytes of shared memory: A's columns of the slice and (by group) their sums, the rings, the partial sums and in clusters the
// CTA's sums (two rounds' of both).
__host__ __device__ constexpr int64_t w4_smem(int groups, int64_t slice, bool cluster)
{
    return slice * 2 * (2048 + 32 * groups) + kW4Warps * (kW4Ahead * 2048 + 1024) + (cluster ? 2 * kW4Round * 512 : 0);
}

// GW: words of eight codes that a lane has of a group (1, 2, 4: groups of 32, 64, 128).
template <typename T, int GW>
__global__ void __launch_bounds__(kW4Threads, 1) w4_kernel(const __grid_constant__ W4Params p)
{
    constexpr int GROUP = 32 * GW, GROUPS = 256 / GROUP;   // groups of a step
    constexpr int OWN = (GROUPS + 3) / 4;                  // of a row's groups, those whose scale and zero a lane brings: t, t + 4
    extern __shared__ uint4 act[];                         // [128 columns][word][lane ^ turn(word)]
    // (turned, so that eight neighbouring lanes write pieces of eight different banks when they lay A out: 4096 x 4096, eight rows 8.1 ->
    // 7.8 us. With smaller groups, where they write two or four, the turn cost more: 65536 x 1024, groups of 64, 18.2 -> 21.5)
    auto turn = [](int word) { return GW == 4 ? 2 * (word & 3) : 0; };
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
    const int cluster = static_cast<int>(blockIdx.x) / ctas, m0 = static_cast<int>(blockIdx.y) * kW4Rows;   // (0 unless K is)
    const int step0 = static_cast<int>(static_cast<int64_t>(p.steps) * rank / ctas);
    const int count = static_cast<int>(static_cast<int64_t>(p.steps) * (rank + 1) / ctas) - step0;
    const int groups = p.K / GROUP, my_groups = groups - step0 * GROUPS;   // of a row, in all and from this slice on
    float *const xsum = reinterpret_cast<float *>(act + p.slice * 256);                        // [group of the slice][row of A]
    uint4 *const rings = reinterpret_cast<uint4 *>(xsum + p.slice * GROUPS * kW4Rows);
    uint4 *const ring = rings + warp * (kW4Ahead * 128) + lane;                                // [slot][128 columns][row g, g + 8] of this lane
    float4 *const reds = reinterpret_cast<float4 *>(rings + kW4Warps * kW4Ahead * 128);        // [round mod 2][warp][lane]
    float4 *const part = reds + 2 * kW4Warps * 32;                                             // [round mod 2][tile of W][lane]
    W4Walk now;
    now.tile = static_cast<int>(static_cast<int64_t>(p.tiles) * cluster / p.clusters);
    now.left = static_cast<int>(static_cast<int64_t>(p.tiles) * (cluster + 1) / p.clusters) - now.tile;
    now.begin(warp, count);
    // ---- the codes of a turn into a slot of the ring, scales and zeros into registers (as they are: whatever used them
    // here would wait for them)
    struct Scales {
        uint16_t s[2][OWN];
        uint8_t z[2][OWN];
    } scales[kW4Ahead];
    W4Walk ahead = now;
    const uint8_t *codes_at[2], *zeros_at[2];   // of this lane's rows, from the slice's first step on
    const uint16_t *scales_at[2];
    auto rows_of_round = [&]() {
        const int row = (ahead.tile + ahead.row_warp(warp)) * 16 + g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = min(row + 8 * h, p.N - 1);   // (rows past the last are not written)
            codes_at[h] = p.codes + r * (p.K / 2) + static_cast<int64_t>(step0) * 128 + 4 * GW * t;
            const int64_t at = r * groups + static_cast<int64_t>(step0) * GROUPS + t;
            scales_at[h] = static_cast<const uint16_t *>(p.scales) + at;
            zeros_at[h] = p.zeros + at;
        }
    };
    rows_of_round();
    const uint32_t ring_at = smem_u32(ring);
    auto load = [&](int slot, Scales &x) {
        if (ahead.turns == 0 && ahead.left > 0) {
            ahead.end_round(warp, count);
            if (ahead.left > 0)
                rows_of_round();
        }
        --ahead.turns;
        const int step = ahead.step, have = my_groups - step * GROUPS;   // groups from this step on
        ahead.step += ahead.warps();
        if (ahead.left > 0 && step < count) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < GROUPS; ++i)
                    if (i < have)   // (past the last group what is there counts with columns of 0)
                        copy_async<4 * GW>(ring_at + (slot * 128u + (i * GW / 4) * 64u + 32u * h) * 16u + 4u * (i * GW % 4),
                                           codes_at[h] + step * 128 + 16 * GW * i);
#pragma unroll
                for (int j = 0; j < OWN; ++j) {
                    x.s[h][j] = 0;
                    x.z[h][j] = 8;
                    if (t + 4 * j < min(GROUPS, have)) {
                        x.s[h][j] = scales_at[h][step * GROUPS + 4 * j];
                        if (p.zeros)
                            x.z[h][j] = zeros_at[h][step * GROUPS + 4 * j];
                    }
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u)
        load(u, scales[u]);
    // ---- A's columns, each piece (eight columns of a row, one lane's word of W) to where the products take it, and the sums of the
    // groups' columns: up to four pieces to a thread with shuffles, for more as products with ones once all are there
    const int rows = min(p.M - m0, kW4Rows);   // (what stands in rows past the last stays in columns of the products that are not written)
    const int k16 = lane % 16, of_lane = GW == 4 ? k16 / 4 : GW == 2 ? k16 / 2 % 4 : k16 % 4;
    const int word = GW == 4 ? k16 % 4 : GW == 2 ? k16 / 8 * 2 + k16 % 2 : k16 / 4;
    using Pair = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
    uint32_t largest = 0;   // |x| of the thread's even and odd columns; NaN stays
    auto lay_out = [&](auto on_their_way, auto with_sums) {
        constexpr int N = decltype(on_their_way)::value;
#pragma unroll 1
        for (W4Pieces at(warp, count); at.row < rows;) {
            uint4 v[N];
            int row[N], piece[N];
#pragma unroll
            for (int u = 0; u < N; ++u, at.next(count)) {
                row[u] = at.row;
                piece[u] = at.piece;
                const int64_t k = (static_cast<int64_t>(step0) + at.piece) * 256 + 8 * lane;
                v[u] = make_uint4(0, 0, 0, 0);
                if (at.row < rows && k < p.K)
                    v[u] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.a) + (m0 + at.row) * p.lda + k);
            }
#pragma unroll
            for (int u = 0; u < N; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x = e == 0 ? v[u].x : e == 1 ? v[u].y : e == 2 ? v[u].z : v[u].w;
                    const Pair y = __hmax2_nan(*reinterpret_cast<const Pair *>(&largest), __habs2(*reinterpret_cast<const Pair *>(&x)));
                    largest = *reinterpret_cast<const uint32_t *>(&y);
                }
                float sum = 0.0f;
                if constexpr (decltype(with_sums)::value) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = unpack2<T>(e == 0 ? v[u].x : e == 1 ? v[u].y : e == 2 ? v[u].z : v[u].w);
                        sum += x.x + x.y;
                    }
#pragma unroll
                    for (int o = GROUP / 16; o > 0; o /= 2)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                }
                if (row[u] < rows) {   // (the word's pairs are columns j and j + 4)
                    const int k8 = piece[u] * 32 + lane;
                    act[(k8 / 16 * 4 + word) * 32 + ((row[u] * 4 + of_lane) ^ turn(word))] =
                        make_uint4(__byte_perm(v[u].x, v[u].z, 0x5410), __byte_perm(v[u].x, v[u].z, 0x7632),
                                   __byte_perm(v[u].y, v[u].w, 0x5410), __byte_perm(v[u].y, v[u].w, 0x7632));
                    if (decltype(with_sums)::value && k8 % (GROUP / 8) == 0)
                        xsum[k8 / (GROUP / 8) * kW4Rows + row[u]] = sum;
                }
            }
        }
    };
    const int pieces = rows * count;
    if (pieces <= 2 * kW4Warps) {
        lay_out(std::integral_constant<int, 2>{}, std::true_type{});
    } else if (pieces <= 4 * kW4Warps) {
        lay_out(std::integral_constant<int, 4>{}, std::true_type{});
    } else {
        lay_out(std::integral_constant<int, 8>{}, std::false_type{});
        __syncthreads();
#pragma unroll 1
        for (int q = warp; q < count * GROUPS; q += kW4Warps) {
            constexpr uint32_t ONES = W4Codes<T>::ONES;
            float sum[4] = {};
#pragma unroll
            for (int w = 0; w < GW; ++w) {
                const uint4 x = act[(q * GW + w) * 32 + (lane ^ turn(w))];
                mma_16x8x16<T>(sum, ONES, ONES, ONES, ONES, x.x, x.z);
                mma_16x8x16<T>(sum, ONES, ONES, ONES, ONES, x.y, x.w);
            }
            if (g == 0)
                *reinterpret_cast<float2 *>(xsum + q * kW4Rows + 2 * t) = make_float2(sum[0], sum[1]);
        }
    }
    const float2 top = unpack2<T>(largest);
    const bool moderate = __syncthreads_and(top.x < W4Codes<T>::LIMIT && top.y < W4Codes<T>::LIMIT);   // (not of NaN)
    // ---- bias, activation and one rounding of a tile of sums (rows g and g + 8 of the tile, rows 2 t and 2 t + 1 of A)
    auto finish = [&](float4 y, int tile) {
        const int row = tile * 16 + g;
        if (p.bias) {
            const T *bias = static_cast<const T *>(p.bias);
            const float b0 = row < p.N ? static_cast<float>(bias[row]) : 0.0f, b1 = row + 8 < p.N ? static_cast<float>(bias[row + 8]) : 0.0f;
            y = make_float4(y.x + b0, y.y + b0, y.z + b1, y.w + b1);
        }
        w4_activate(p.epilogue, y.x, y.y);
        w4_activate(p.epilogue, y.z, y.w);
        // lanes of even g take token 2 t of rows g and g + 1, those of odd g token 2 t + 1: two rows to a store
        const bool odd = g & 1;
        const float a = __shfl_xor_sync(0xffffffffu, odd ? y.x : y.y, 4), b = __shfl_xor_sync(0xffffffffu, odd ? y.z : y.w, 4);
        const uint32_t lo = odd ? pack2<T>(a, y.y) : pack2<T>(y.x, a), hi = odd ? pack2<T>(b, y.w) : pack2<T>(y.z, b);
        const int m = m0 + 2 * t + odd, first = row & ~1;
        if (m < p.M) {
            T *dst = static_cast<T *>(p.c) + m * p.ldc + first;
            if (first < p.N)
                *reinterpret_cast<uint32_t *>(dst) = lo;
            if (first + 8 < p.N)
                *reinterpret_cast<uint32_t *>(dst + 8) = hi;
        }
    };
    for (int buf = 0; now.left > 0; now.end_round(warp, count), buf ^= 1) {
        const int row_warp = now.row_warp(warp), k_warp = warp >> now.log_rows, k_warps = now.warps();
        float acc[4] = {};
        // codes of the turn's step (in slot `slot`) times A's columns
        auto products = [&](int slot, int step, const Scales &mine, auto all_moderate) {
            constexpr bool MODERATE = decltype(all_moderate)::value;
            const uint4 *b = act + step * 256;
            const float *xs = xsum + step * (GROUPS * kW4Rows) + 2 * t;
            // s (UNIT sum + ODD_UNIT odd - (BASE + z) xsum), the unit with the scale
            constexpr float PER_ODD = W4Codes<T>::ODD_UNIT / W4Codes<T>::UNIT;
            float s[2][OWN], z[2][OWN];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < OWN; ++j) {
                    const float zero = static_cast<float>(mine.z[h][j] & 15);
                    s[h][j] = unpack2<T>(mine.s[h][j]).x * (MODERATE ? W4Codes<T>::UNIT : 1.0f);
                    z[h][j] = MODERATE ? (W4Codes<T>::BASE + zero) * (-1.0f / W4Codes<T>::UNIT) : zero;
                }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 w0 = ring[slot * 128 + half * 64], w1 = ring[slot * 128 + half * 64 + 32];
                const uint32_t codes[2][4] = {{w0.x, w0.y, w0.z, w0.w}, {w1.x, w1.y, w1.z, w1.w}};
#pragma unroll
                for (int i = half * (GROUPS / 2); i < (half + 1) * (GROUPS / 2); ++i) {
                    float sum[4] = {}, odd[4] = {};
                    const int from = (lane & ~3) | (i & 3);
                    const float s0 = __shfl_sync(0xffffffffu, s[0][i / 4], from), s1 = __shfl_sync(0xffffffffu, s[1][i / 4], from);
                    const float z0 = __shfl_sync(0xffffffffu, z[0][i / 4], from), z1 = __shfl_sync(0xffffffffu, z[1][i / 4], from);
#pragma unroll
                    for (int w = i * GW; w < (i + 1) * GW; ++w) {   // of the step's eight words
                        uint32_t a0[4], a1[4];
                        if constexpr (MODERATE) {
                            W4Codes<T>::unpack(codes[0][w % 4], a0);
                            W4Codes<T>::unpack(codes[1][w % 4], a1);
                        } else {
                            w4_unpack_minus_zero<T>(codes[0][w % 4], static_cast<uint32_t>(z0), a0);
                            w4_unpack_minus_zero<T>(codes[1][w % 4], static_cast<uint32_t>(z1), a1);
                        }
                        const uint4 x = b[w * 32 + (lane ^ turn(w))];
                        mma_16x8x16<T>(sum, a0[0], a1[0], a0[2], a1[2], x.x, x.z);
                        mma_16x8x16<T>(odd, a0[1], a1[1], a0[3], a1[3], x.y, x.w);
                    }
                    if constexpr (MODERATE) {
                        const float2 x = *reinterpret_cast<const float2 *>(xs + i * kW4Rows);
                        acc[0] = fmaf(fmaf(z0, x.x, fmaf(odd[0], PER_ODD, sum[0])), s0, acc[0]);
                        acc[1] = fmaf(fmaf(z0, x.y, fmaf(odd[1], PER_ODD, sum[1])), s0, acc[1]);
                        acc[2] = fmaf(fmaf(z1, x.x, fmaf(odd[2], PER_ODD, sum[2])), s1, acc[2]);
                        acc[3] = fmaf(fmaf(z1, x.y, fmaf(odd[3], PER_ODD, sum[3])), s1, acc[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[e] = fmaf((sum[e] + odd[e]) * (e < 2 ? s0 : s1), MINUS_ZERO_UNIT<T>, acc[e]);
                    }
                }
            }
        };
        for (int turn = 0; turn < now.turns; turn += kW4Ahead) {
#pragma unroll
            for (int u = 0; u < kW4Ahead; ++u) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kW4Ahead - 1) : "memory");   // (a lane reads only what it has copied)
                const int step = now.step + (turn + u) * k_warps;
                if (step < count) {
                    if (moderate)
                        products(u, step, scales[u], std::true_type{});
                    else
                        products(u, step, scales[u], std::false_type{});
                }
                load(u, scales[u]);
            }
        }
        // ---- the round's sums: the warps of a tile, then the CTAs, in order. One barrier, after which the others go on: where they
        // write in the next round nothing is read any more, since who reads passes that barrier first.
        float4 *const red = reds + buf * (kW4Warps * 32);
        if (k_warp > 0)
            red[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        if (k_warp == 0) {
            float4 y = make_float4(acc[0], acc[1], acc[2], acc[3]);
            for (int k = 1; k < k_warps; ++k) {
                const float4 v = red[(warp + (k << now.log_rows)) * 32 + lane];
                y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
            }
            if (ctas == 1)
                finish(y, now.tile + row_warp);
            else
                part[(buf * kW4Round + row_warp) * 32 + lane] = y;
        }
        if (ctas > 1) {
            cluster_sync();
            const int f = warp * ctas + rank;   // one tile at most: the round has no more than kW4Round
            if (f < 1 << now.log_rows) {
                float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int c = 0; c < ctas; ++c) {
                    const float4 v =
                        ld_shared_cluster_f4(mapa_shared(smem_u32(part + (buf * kW4Round + f) * 32 + lane), static_cast<uint32_t>(c)));
                    y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
                }
                finish(y, now.tile + f);
            }
        }
    }
    if (ctas > 1)
        cluster_sync();   // the other CTAs have read this one's sums
}

}  // namespace gb300
