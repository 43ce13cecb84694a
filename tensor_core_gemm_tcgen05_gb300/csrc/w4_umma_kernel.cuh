// The product of w4_kernel.cuh for more rows of A, on the fifth-generation tensor cores: W's tile is the
// operand in Tensor Memory (128 rows of W, a lane each), A's columns come by TMA, and the sum of every group lies in
// Tensor Memory until it is scaled, so that as there no weight is rounded.
//
// A step is 128 columns of W, a block eight steps. One CTA to an SM; a cluster of CTAs shares the columns of a tile. Roles:
//  * producer: TMA, a step's codes (64 bytes of each row) and A's columns into a ring of stages;
//  * six loaders: a block's scales and zeros, read along the rows of W (a thread for each row, step by step,
//    touches a line per row and step) and laid out by group;
//  * four or two groups of four warps, a row of W per thread, take the codes of steps in turn to Tensor Memory as code - zero
//    (pairs of consecutive columns, the lower in the low half, as the product wants them), and a thread of each issues
//    the step's products: several issuers, since one thread's waits and instructions took longer than the products;
//  * one or two groups of four warps scale and add up the sums of the groups, a row of W per thread.
// Every wait is bounded.
//
// Measured (captured, weights from HBM; 5.2 us at the copy rate): 16384 x 4096, groups of 128, 16 rows 16.9 us, 64 rows 21.4; 4096 x 16384,
// groups of 64 in BF16, 64 rows 29.3. What bounds it is the way of a step from group to group, none of its parts alone: of the
// last, without the loads of weights 27.2, with one product of eight 26.3, without unpacking 27.0, without the loads of scales
// 27.9, without scaling 29.3, without all but the first 22.6. Tried at 16384 x 4096, 16 rows: two CTAs to an SM, roles merged, 17.5; one
// issuer and six buffers of codes 22.8; three groups with two buffers 18.9; five groups 16.6 (but 32 rows 18.1 -> 20.1); halves of
// a step handed over one by one 18.3.
#pragma once

#include "w4_kernel.cuh"

namespace gb300 {

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Waits for the loads issued before and ties their registers to this point.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(r[i]));
}

// TOK: rows of A (tokens) of a CTA, 16, 32 or 64. GROUP: columns to a scale.
template <typename T_, int TOK_, int GROUP_>
struct W4UmmaConfig {
    using T = T_;
    static constexpr int TOK = TOK_, GROUP = GROUP_;
    static constexpr int GROUPS = 128 / GROUP;   // of a step
    static constexpr int CODES = 128 * 64, ACT_ATOM = TOK * 128, STAGE = CODES + 2 * ACT_ATOM;
    static constexpr int STAGES = TOK == 64 ? 7 : TOK == 32 ? 10 : 14;
    // a block's scales (16 bits) and zeros (8 bits), by group
    static constexpr int BLOCK = 8, BLOCK_GROUPS = BLOCK * GROUPS, SCALE_PITCH = 130, ZERO_PITCH = 132;
    static constexpr int SCALES = BLOCK_GROUPS * SCALE_PITCH * 2, ZEROS = BLOCK_GROUPS * ZERO_PITCH;
    static constexpr int SCALE_OFF = STAGES * STAGE, ZERO_OFF = SCALE_OFF + 2 * SCALES;
    // Tensor Memory: of each unpacking group the codes of a step or two (64 columns each, 16-bit pairs), then its sums
    static constexpr bool MANY_SUMS = TOK * GROUPS > 64;
    static constexpr int UNPACKERS = MANY_SUMS ? 2 : 4, CODE_BUFS = MANY_SUMS ? 2 : 1, SUM_COLS = MANY_SUMS ? 128 : 64;
    static constexpr int D_COL = UNPACKERS * CODE_BUFS * 64, TMEM_COLS = 512;
    // A commit costs as much as three of these products (164 cycles, 56 each), so there is one for as many groups (a batch) as
    // have their sums side by side.
    static constexpr int ROOM = SUM_COLS / TOK, BATCH = GROUPS < ROOM ? GROUPS : ROOM, BATCHES = GROUPS / BATCH, SLOTS = ROOM / BATCH;
    static_assert(SLOTS * BATCH == ROOM && BATCHES * BATCH == GROUPS, "powers of two");
    static_assert(D_COL + UNPACKERS * SUM_COLS <= TMEM_COLS, "Tensor Memory columns");
    static constexpr int PITCH = 132;   // of the partial sums, in floats
    static constexpr int NUM_BARS = 2 * STAGES + (2 + CODE_BUFS + 2 * SLOTS) * UNPACKERS + 4;
    static constexpr int BAR_OFF = (ZERO_OFF + 2 * ZEROS + 7) / 8 * 8;
    static constexpr int SMEM_BYTES = 1024 + BAR_OFF + NUM_BARS * 8 + 16;
    static constexpr int UNPACK_WARPS = 4 * UNPACKERS, SCALE_WARPS = TOK == 64 ? 8 : 4, SCALE_TOK = TOK * 4 / SCALE_WARPS;
    static constexpr int PRODUCER_WARP = UNPACK_WARPS + SCALE_WARPS, LOADER_WARP = PRODUCER_WARP + 1;
    static constexpr int LOADERS = 3;   // warps, of scales and of zeros each
    static constexpr int NUM_THREADS = 32 * (LOADER_WARP + 2 * LOADERS);
    static_assert(SMEM_BYTES + 1024 <= 233472, "shared memory of an SM");
    static_assert(TOK * PITCH * 4 <= SCALE_OFF, "the partial sums lie over the stages");
    static constexpr uint32_t TYPE_BITS = std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
    // FP32 sums, M = 128, N = TOK, both operands K-major
    static constexpr uint32_t IDESC = (1u << 4) | TYPE_BITS | (static_cast<uint32_t>(TOK >> 3) << 17) | (128u >> 4 << 24);
};

// Codes 2 i and 2 i + 1 of a word, minus zero, as pair i of x, times a power of two. A byte under zeros is a subnormal number of the
// type, its value times the smallest one: the even code, or 16 times the odd one. One exact multiply-add brings both to
// the same power of two and takes the zero. What makes up for it goes to the scales (OF_SCALE) and the result (OF_RESULT).
//  * FP16: 2^-9; the scales are below 2^16.
//  * BF16: 2^-11, so that a group's sum (128 times 15 at most) stays in FP32's range whatever is multiplied, and all of it to the result,
//    since scales may be of any size. (The scales' half keeps registers as they were: without a product there the
//    compiler spilled 216 bytes, 64 rows of 4096 x 4096 in groups of 32 16.6 us for 15.9.)
template <typename T>
struct W4Pairs;
template <>
struct W4Pairs<__half> {
    static constexpr float OF_SCALE = 512.0f, OF_RESULT = 1.0f;   // 2^-24 2^15 = 2^-9
    __half2 minus;
    __device__ __forceinline__ explicit W4Pairs(uint32_t zero)
    {
        const uint32_t v = zero * 0x10001u, times = 0xf800f800u;   // -2^15
        minus = __hmul2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&times));
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t v) const
    {
        const uint32_t times = 0x68007800u;   // 2^15, 2^11
        const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&times), minus);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
};
template <>
struct W4Pairs<__nv_bfloat16> {
    static constexpr float OF_SCALE = 0.5f, OF_RESULT = 4096.0f;   // 2^-133 2^122 = 2^-11
    __nv_bfloat162 minus;
    __device__ __forceinline__ explicit W4Pairs(uint32_t zero)
    {
        const uint32_t v = zero * 0x10001u, times = 0xfc80fc80u;   // -2^122
        minus = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&times));
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t v) const
    {
        const uint32_t times = 0x7a807c80u;   // 2^122, 2^118
        const __nv_bfloat162 y =
            __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&times), minus);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
};

template <typename T>
__device__ __forceinline__ void w4_unpack(const W4Pairs<T> &pairs, uint32_t w, uint32_t *x)
{
    const uint32_t even = w & 0x0f0f0f0fu, odd = w & 0xf0f0f0f0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // byte i of either, each under the sign (selector + 8) of an even byte: 0
        uint32_t v;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(even), "r"(odd), "r"(0x8480u + 0x0101u * i));
        x[i] = pairs(v);
    }
}

// The partial sums of a cluster's CTAs, each part[token * pitch + row of W], added up in the order of the CTAs, and this
// CTA's share of the outputs written: bias, activation, one rounding. All threads of all its CTAs call it, after a barrier.
template <typename T>
__device__ __forceinline__ void w4_finish(const W4Params &p, const float *part, int pitch, int rows, int tokens, int n0, int m0,
                                          int rank, int ctas)
{
    if (ctas > 1)
        cluster_sync();
    const int pairs = tokens * rows / 2, share = (pairs + ctas - 1) / ctas;   // pairs of rows of W for one token
    const uint32_t base = smem_u32(part);
    for (int i = rank * share + static_cast<int>(threadIdx.x); i < min(pairs, (rank + 1) * share); i += static_cast<int>(blockDim.x)) {
        const int m = i / (rows / 2), r = i % (rows / 2) * 2;
        if (m0 + m >= p.M || n0 + r >= p.N)
            continue;
        float2 y = make_float2(0.0f, 0.0f);
        if (ctas == 1) {   // (shared::cluster addresses only come from mapa, in a cluster)
            y = *reinterpret_cast<const float2 *>(part + m * pitch + r);
        } else {
            for (int c = 0; c < ctas; ++c) {
                const float2 v = ld_shared_cluster_f2(mapa_shared(base + static_cast<uint32_t>(m * pitch + r) * 4u, static_cast<uint32_t>(c)));
                y.x += v.x;
                y.y += v.y;
            }
        }
        if (p.bias) {
            const float2 b = unpack2<T>(*reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.bias) + n0 + r));
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

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NUM_THREADS, 1)
    w4_umma_kernel(const __grid_constant__ CUtensorMap tmap_codes, const __grid_constant__ CUtensorMap tmap_a,
                   const __grid_constant__ W4Params p)
{
    using T = typename Cfg::T;
    constexpr int TOK = Cfg::TOK, GROUPS = Cfg::GROUPS, STAGES = Cfg::STAGES, SLOTS = Cfg::SLOTS, UNPACKERS = Cfg::UNPACKERS;
    constexpr int BATCH = Cfg::BATCH, BATCHES = Cfg::BATCHES, CODE_BUFS = Cfg::CODE_BUFS;
    constexpr int BLOCK = Cfg::BLOCK;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sp = smem_raw + (base - raw);
    const uint32_t full0 = base + Cfg::BAR_OFF, empty0 = full0 + 8u * STAGES, a_full0 = empty0 + 8u * STAGES;
    const uint32_t drain0 = a_full0 + 8u * UNPACKERS, a_done0 = drain0 + 8u * UNPACKERS, d_full0 = a_done0 + 8u * UNPACKERS * CODE_BUFS, d_empty0 = d_full0 + 8u * UNPACKERS * SLOTS;
    const uint32_t s_full0 = d_empty0 + 8u * UNPACKERS * SLOTS, s_empty0 = s_full0 + 16u;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sp + Cfg::BAR_OFF + Cfg::NUM_BARS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full0 + 8u * i, 1);
            mbar_init(empty0 + 8u * i, Cfg::SCALE_WARPS);
        }
        for (int i = 0; i < UNPACKERS; ++i) {
            mbar_init(a_full0 + 8u * i, 4);
            mbar_init(drain0 + 8u * i, 1);
        }
        for (int i = 0; i < UNPACKERS * CODE_BUFS; ++i)
            mbar_init(a_done0 + 8u * i, 1);
        for (int i = 0; i < UNPACKERS * SLOTS; ++i) {
            mbar_init(d_full0 + 8u * i, 1);
            mbar_init(d_empty0 + 8u * i, Cfg::SCALE_WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8u * i, 2 * Cfg::LOADERS);
            mbar_init(s_empty0 + 8u * i, Cfg::UNPACK_WARPS + Cfg::SCALE_WARPS);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_codes);
        tma_prefetch_desc(&tmap_a);
    }
    if (warp == Cfg::PRODUCER_WARP) {
        tmem_alloc<1>(smem_u32(tmem_slot), Cfg::TMEM_COLS);
        tmem_relinquish<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    grid_dependency_wait();   // nothing above touched global memory
    grid_dependents_launch();
    const uint32_t tmem = *tmem_slot;
    const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
    const int n0 = static_cast<int>(blockIdx.x) / ctas * 128, m0 = static_cast<int>(blockIdx.y) * TOK;
    const int step0 = static_cast<int>(static_cast<int64_t>(p.steps) * rank / ctas);
    const int count = static_cast<int>(static_cast<int64_t>(p.steps) * (rank + 1) / ctas) - step0;
    const int groups = p.K / Cfg::GROUP;
    const WaitCtl wc{abort_flag, p.err, p.timeout_ns};
    const int quarter = warp & 3, row = quarter * 32 + lane;   // of the tile: of the warps with rows
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float acc[Cfg::SCALE_TOK] = {};

    if (warp == Cfg::PRODUCER_WARP) {
        if (lane == 0) {
            bool ok = true;
            int issued = 0;
            for (int i = 0; ok && i < count; ++i) {
                const uint32_t stage = static_cast<uint32_t>(i % STAGES), at = base + stage * Cfg::STAGE, full = full0 + 8u * stage;
                if (!(ok = wait_bounded(empty0 + 8u * stage, (static_cast<uint32_t>(i / STAGES) & 1u) ^ 1u, wc, ERR_PRODUCER_SLOT)))
                    break;
                if (p.debug & DEBUG_WITHHOLD_FIRST_LOAD)   // test hook: never loaded
                    break;
                mbar_arrive_expect_tx(full, Cfg::STAGE);
                tma_load_2d(at, &tmap_codes, full, (step0 + i) * 64, n0);
                tma_load_2d(at + Cfg::CODES, &tmap_a, full, (step0 + i) * 128, m0);
                tma_load_2d(at + Cfg::CODES + Cfg::ACT_ATOM, &tmap_a, full, (step0 + i) * 128 + 64, m0);
                ++issued;
            }
            if (!ok)   // let every copy started land before the stages are written over
                for (int i = max(0, issued - STAGES); i < issued; ++i)
                    wait_until(full0 + 8u * static_cast<uint32_t>(i % STAGES), static_cast<uint32_t>(i / STAGES) & 1u, p.timeout_ns, p.err);
        }
    } else if (warp >= Cfg::LOADER_WARP) {
        // ---- scales (the first loaders) and zeros: lanes along the groups of a row, a few rows to a load, the loads
        // dealt to the loaders, a batch in flight (without branches: those would wait for each load)
        const bool zero = warp >= Cfg::LOADER_WARP + Cfg::LOADERS;
        constexpr int WIDE = Cfg::BLOCK_GROUPS, ROWS = 32 / WIDE, LOADS = 128 / ROWS, BATCH = 16;
        static_assert(WIDE <= 32, "a lane for each group of a block");
        const int e = lane % WIDE, loader = warp - Cfg::LOADER_WARP - (zero ? Cfg::LOADERS : 0);
        const int last = p.N - 1 - n0;   // (rows past it are not written)
        auto copy = [&](auto *src, auto *dst, int pitch, int at, bool on, uint32_t none) {
            using V = std::remove_pointer_t<decltype(dst)>;
            src += static_cast<int64_t>(n0) * groups + at;
            for (int k0 = loader; k0 < LOADS; k0 += Cfg::LOADERS * BATCH) {
                V v[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int r = (k0 + k * Cfg::LOADERS) * ROWS + lane / WIDE;
                    v[k] = static_cast<V>(none);
                    if (on && r < 128)
                        v[k] = src[static_cast<int64_t>(min(r, last)) * groups];
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int r = (k0 + k * Cfg::LOADERS) * ROWS + lane / WIDE;
                    if (r < 128)
                        dst[e * pitch + r] = v[k];
                }
            }
        };
        bool ok = true;
        for (int b = 0; ok && b * BLOCK < count; ++b) {
            const uint32_t slot = static_cast<uint32_t>(b & 1);
            if (b >= 2 && !(ok = wait_warp(s_empty0 + 8u * slot, static_cast<uint32_t>((b >> 1) - 1) & 1u, wc, ERR_PRODUCER_SLOT, lane)))
                break;
            const int at = (step0 + b * BLOCK) * GROUPS + e;
            const bool on = at < groups && b * BLOCK + e / GROUPS < count;
            if (zero)
                copy(p.zeros, sp + Cfg::ZERO_OFF + slot * Cfg::ZEROS, Cfg::ZERO_PITCH, at, on && p.zeros, 8u);
            else
                copy(static_cast<const uint16_t *>(p.scales), reinterpret_cast<uint16_t *>(sp + Cfg::SCALE_OFF + slot * Cfg::SCALES),
                     Cfg::SCALE_PITCH, at, on, 0u);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(s_full0 + 8u * slot);
        }
    } else if (warp < Cfg::UNPACK_WARPS) {
        // ---- codes of the steps w, w + 4, ..., and their products
        const int w = warp >> 2;
        const uint32_t codes0 = tmem + 64u * static_cast<uint32_t>(w * CODE_BUFS), full_w = d_full0 + 8u * static_cast<uint32_t>(w * SLOTS);
        const uint32_t empty_w = d_empty0 + 8u * static_cast<uint32_t>(w * SLOTS);
        bool ok = true;
        for (int i = w, t = 0; i < count; i += UNPACKERS, ++t) {
            const uint32_t stage = static_cast<uint32_t>(i % STAGES), block = static_cast<uint32_t>(i / BLOCK & 1);
            const uint32_t buf = static_cast<uint32_t>(t % CODE_BUFS), codes = codes0 + 64u * buf;
            const uint32_t a_done = a_done0 + 8u * (static_cast<uint32_t>(w * CODE_BUFS) + buf);
            // the products that read this part of Tensor Memory before are over
            if (t >= CODE_BUFS)
                ok = wait_warp(a_done, static_cast<uint32_t>(t / CODE_BUFS - 1) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane);
            ok = ok && wait_warp(s_full0 + 8u * block, static_cast<uint32_t>(i / (2 * BLOCK)) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane) &&
                 wait_warp(full0 + 8u * stage, static_cast<uint32_t>(i / STAGES) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane);
            if (!ok)
                break;
            tc_fence_after_sync();
            const uint8_t *src = sp + stage * Cfg::STAGE + row * 64;
            const uint8_t *zeros = sp + Cfg::ZERO_OFF + block * Cfg::ZEROS + i % BLOCK * GROUPS * Cfg::ZERO_PITCH + row;
            uint4 v[4];   // 32 codes each (the 64-byte swizzle: piece c at c ^ (row / 2 mod 4)), all read before the first store
            uint32_t zero[GROUPS];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = *reinterpret_cast<const uint4 *>(src + ((c ^ ((row >> 1) & 3)) << 4));
#pragma unroll
            for (int e = 0; e < GROUPS; ++e)
                zero[e] = zeros[e * Cfg::ZERO_PITCH] & 15u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const W4Pairs<T> pairs(zero[c * GROUPS / 4]);
                uint32_t x[16];
                w4_unpack(pairs, v[c].x, x);
                w4_unpack(pairs, v[c].y, x + 4);
                w4_unpack(pairs, v[c].z, x + 8);
                w4_unpack(pairs, v[c].w, x + 12);
                tmem_st_32x32b_x16(codes + (static_cast<uint32_t>(quarter * 32) << 16) + 16u * c, x);
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(a_full0 + 8u * static_cast<uint32_t>(w));
                if (i % BLOCK >= BLOCK - UNPACKERS)   // its last step of the block
                    mbar_arrive(s_empty0 + 8u * block);
            }
            if (quarter == 0 && lane == 0) {
                ok = wait_bounded(a_full0 + 8u * static_cast<uint32_t>(w), static_cast<uint32_t>(t) & 1u, wc, ERR_MMA_OPERANDS);
                const uint64_t b = sw128_desc(base + stage * Cfg::STAGE + Cfg::CODES, 16, 1024);
#pragma unroll
                for (int batch = 0; batch < BATCHES; ++batch) {
                    const int j = t * BATCHES + batch;
                    const uint32_t slot = static_cast<uint32_t>(j % SLOTS);
                    if (ok && j >= SLOTS)
                        ok = wait_bounded(empty_w + 8u * slot, static_cast<uint32_t>(j / SLOTS - 1) & 1u, wc, ERR_MMA_ACCUMULATOR);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int k = 0; k < BATCH * Cfg::GROUP / 16; ++k) {
                        constexpr int PER = Cfg::GROUP / 16;
                        const int kk = batch * BATCH * PER + k;
                        umma_f16_tmem_a(tmem + Cfg::D_COL + static_cast<uint32_t>(w * Cfg::SUM_COLS) + (slot * BATCH + k / PER) * TOK, codes + 8u * kk,
                                        b + static_cast<uint64_t>(((kk >> 2) * Cfg::ACT_ATOM + (kk & 3) * 32) >> 4), Cfg::IDESC,
                                        k % PER > 0 ? 1u : 0u);
                    }
                    umma_commit(full_w + 8u * slot);
                }
                if (ok)
                    umma_commit(a_done);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);   // (the first warp's; another's own)
            if (!ok)
                break;
        }
        if (!ok && quarter == 0 && lane == 0) {   // let the products issued end before the stages are written over
            umma_commit(drain0 + 8u * static_cast<uint32_t>(w));
            wait_until(drain0 + 8u * static_cast<uint32_t>(w), 0, p.timeout_ns, p.err);
        }
        __syncwarp();
    } else {
        // ---- sums of the groups, this half (or all) of the tokens
        const int part = (warp - Cfg::UNPACK_WARPS) >> 2;
        bool ok = true;
        for (int i = 0; ok && i < count; ++i) {
            const uint32_t block = static_cast<uint32_t>(i / BLOCK & 1);
            if (i % BLOCK == 0 &&
                !(ok = wait_warp(s_full0 + 8u * block, static_cast<uint32_t>(i / (2 * BLOCK)) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane)))
                break;
            const uint16_t *scales = reinterpret_cast<const uint16_t *>(sp + Cfg::SCALE_OFF + block * Cfg::SCALES) +
                                     i % BLOCK * GROUPS * Cfg::SCALE_PITCH + row;
#pragma unroll
            for (int batch = 0; batch < BATCHES; ++batch) {
                const int j = i / UNPACKERS * BATCHES + batch;   // of the unpacking group's
                const uint32_t slot = static_cast<uint32_t>(i % UNPACKERS * SLOTS + j % SLOTS);
                if (!(ok = wait_warp(d_full0 + 8u * slot, static_cast<uint32_t>(j / SLOTS) & 1u, wc, ERR_EPILOGUE_ACCUMULATOR, lane)))
                    break;
                tc_fence_after_sync();
#pragma unroll
                for (int e = 0; e < BATCH; ++e) {
                    const float s = unpack2<T>(scales[(batch * BATCH + e) * Cfg::SCALE_PITCH]).x * W4Pairs<T>::OF_SCALE;
                    const uint32_t at = lanes + Cfg::D_COL + static_cast<uint32_t>(i % UNPACKERS * Cfg::SUM_COLS + (j % SLOTS * BATCH + e) * TOK + part * Cfg::SCALE_TOK);
#pragma unroll
                    for (int t0 = 0; t0 < Cfg::SCALE_TOK; t0 += 16) {
                        uint32_t d[16];
                        tmem_ld_32x32b_x16(at + static_cast<uint32_t>(t0), d);
                        tmem_ld_wait_for(d);
                        if (e + 1 == BATCH && t0 + 16 == Cfg::SCALE_TOK) {
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(d_empty0 + 8u * slot);
                        }
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            acc[t0 + t] = fmaf(__uint_as_float(d[t]), s, acc[t0 + t]);
                    }
                }
            }
            if (!ok)
                break;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(empty0 + 8u * static_cast<uint32_t>(i % STAGES));   // the step's products are over: nothing reads its stage
                if (i % BLOCK == BLOCK - 1)
                    mbar_arrive(s_empty0 + 8u * block);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == Cfg::PRODUCER_WARP) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, Cfg::TMEM_COLS);
    }
    // every stage has been read: the partial sums go over them
    float *sums = reinterpret_cast<float *>(sp);
    if (warp >= Cfg::UNPACK_WARPS && warp < Cfg::PRODUCER_WARP) {
        const int part = (warp - Cfg::UNPACK_WARPS) >> 2;
#pragma unroll
        for (int t = 0; t < Cfg::SCALE_TOK; ++t)
            sums[(part * Cfg::SCALE_TOK + t) * Cfg::PITCH + row] = acc[t] * W4Pairs<T>::OF_RESULT;   // (of the final sums: 64 rows of 16384 x 4096 in BF16 21.3 us -> 21.5)
    }
    __syncthreads();
    w4_finish<T>(p, sums, Cfg::PITCH, 128, TOK, n0, m0, rank, ctas);
}

}  // namespace gb300
