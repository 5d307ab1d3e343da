// w4a16_gate_up_tc.cuh -- h = act(x Wg^T) * (x Wu^T) from int4 weights on
// the 5th-generation tensor cores, for projections wide enough to give every
// multiprocessor a tile of its own.
//
// A tile is `cols` columns (128 at most) of the result: as many gate rows and
// the same up rows, each an M = 128 operand with an accumulator of its own.
// The two accumulators hold a column's gate and up sums in the same
// tensor-memory lane.  `cols` is chosen on the host so that the tiles divide
// evenly over the multiprocessors: no tile is split, nothing is added up
// between blocks, and lanes past `cols` idle.
//
// The levels are exact in bf16 and so is x: a 128-column group's products are
// summed in fp32 by the tensor cores in an accumulator of the group's own,
// and each group's sum is multiplied by its scale and added in fp32
// registers, as in w4a16_gemm.  The gate and up sums are not rounded before
// the activation and the product.
//
// Roles (29 warps), for the gate half (p = 0) and the up half (p = 1):
//  * warps 8 p .. 8 p + 7, levels: four for a stage's first group, four for
//    its second.  A thread is a weight row; it reads the group's 64 packed
//    bytes from the stage and writes 128 bf16 levels to its tensor-memory
//    lane of the group's A slot;
//  * warps 16 + 4 p .. 19 + 4 p, sums: a thread is a row; it reads the
//    group's sums for all tokens and adds them, scaled; at the tile's end the
//    up sums go through shared memory to the gate's threads, which write h;
//  * warps 24 + 2 p and 25 + 2 p, products of p for a stage's first and second
//    group: eight M128 N K16 a group;
//  * warp 28, copies: stages of two groups of the packed rows (two boxes of
//    128-byte rows) and of x (four boxes of 64 columns), as tensor copies.
//
// A nibble becomes a bf16 level by one fma from where it stands in its word
// (gt_levels); that leaves a word's levels in the order (0, 4) (1, 5) (2, 6)
// (3, 7), so x's 16-byte pieces are put in that order in the stage, by the
// level warps.  (Levels in x's own order take a byte permutation each: 29.7
// instead of 26.7 us.)
//
// What bounds it: instructions and hand-offs, not HBM.  F 17,408, K 5,120:
// 1 / 16 / 32 tokens 21.5 / 22.1 / 26.6 us, 4.3 / 4.2 / 3.5 TB/s of weights
// (13.5 us at the copy's rate), of which the hand-offs, sums and copies alone
// take 15.1 / 16.9 / 22.6 and forming the levels the rest.  Measured on the
// way at 32 tokens: one product warp a half and one A fill for two groups
// 34.7; the products of a group and their commits from one elected lane 31.8;
// barriers by running positions instead of divisions 29.4; levels by one fma
// 28.4; a product warp for each half and group 26.7.  Without gain: three A
// slots a half, x copied once for a pair of blocks (28.5 for 28.4).
#pragma once

#include "sv_ptx.cuh"
#include "tc_ops.cuh"
#include "w4a16_gate_up.cuh"

namespace sv {

constexpr int GT_ROWS = 128;                    // lanes of a half's tile
constexpr int GT_GROUPS = 2;                    // of a stage; a half has an A slot and two accumulators for each
constexpr int GT_SUM_WARP = 16, GT_MMA_WARP = 24, GT_COPY_WARP = 28;
constexpr int GT_THREADS = 29 * 32;
constexpr int GT_W_BYTES = GT_ROWS * 128;       // a half's rows of a stage
constexpr int GT_TMEM = 512;                    // columns; 256 of each half: two A slots of 64, four sums of 32

// Shared memory for N tokens (16 or 32): stages, the up sums, barriers.
template <int N>
struct GtSmem {
    static constexpr int STAGES = N == 32 ? 4 : 5;
    static constexpr int X = 2 * GT_W_BYTES, STAGE = X + 4 * N * 128;
    static constexpr int UP = STAGES * STAGE;   // [N][GT_ROWS] fp32
    static constexpr int BARS = UP + N * GT_ROWS * 4;
    // barriers of the stages, then of each half's groups
    static constexpr int FULL = 0, EMPTY = STAGES, A_FULL = 2 * STAGES, A_EMPTY = A_FULL + 4, S_FULL = A_EMPTY + 4,
                         S_EMPTY = S_FULL + 8, X_FULL = S_EMPTY + 8, COUNT = X_FULL + 4;
    static constexpr int BYTES = BARS + 8 * COUNT + 16;
};

struct GateUpTcParams {
    const uint16_t *scales;                     // [2F][G]
    uint16_t *h;                                // [T][F]
    int T, G, F;
    int cols, tiles;                            // columns of a tile; ceil(F / cols)
    int act;
    int *err;
};

// Word of eight levels, k = 0 in the low nibble, to the pairs (0, 4) (1, 5)
// (2, 6) (3, 7), each level as (n - 8) / 64.  A nibble at bits 0..3 or 4..7
// of a bf16 with zeros elsewhere is n 2^-133 or n 2^-129 (subnormals and the
// first normals are evenly spaced), so one shift a word will do and the fma
// moves the nibble: its factor 2^127 or 2^123 is exact, and so is the sum.
__device__ __forceinline__ uint32_t gt_level2(uint32_t nibbles, uint32_t factor)
{
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(nibbles), "r"(factor), "r"(0xBE00BE00u));
    return r;
}

__device__ __forceinline__ void gt_levels(uint32_t w, uint32_t *out)
{
    const uint32_t v = w >> 8;
    out[0] = gt_level2(w & 0x000F000Fu, 0x7F007F00u);
    out[1] = gt_level2(w & 0x00F000F0u, 0x7D007D00u);
    out[2] = gt_level2(v & 0x000F000Fu, 0x7F007F00u);
    out[3] = gt_level2(v & 0x00F000F0u, 0x7D007D00u);
}
constexpr float GT_LEVEL_SCALE = 64.f;

// The eight products of a group (D = A B, M128 N K128) and their hand-offs
// from one elected lane of the warp: the A slot is free, the sums are there,
// the group's x has been read.  b: descriptor of the
// group's first 64 columns, whose K steps are 32 bytes apart; the other 64
// are a box of N rows further.
template <int N>
__device__ __forceinline__ void gt_products(uint32_t d, uint32_t a, uint64_t b, uint32_t slot, uint32_t sums, uint32_t stage)
{
    constexpr uint64_t BOX = N * 128 >> 4;
    asm volatile("{\n\t.reg .pred e, f, t;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 f, %17, %17;\n\t"
                 "setp.eq.b32 t, %17, %17;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %9, %17, f;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %10, %17, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %11, %17, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %12, %17, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %13, %17, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%6], %14, %17, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %15, %17, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%8], %16, %17, t;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%18];\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%19];\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%20];\n\t}"
                 ::"r"(d), "r"(a), "r"(a + 8u), "r"(a + 16u), "r"(a + 24u), "r"(a + 32u), "r"(a + 40u), "r"(a + 48u),
                   "r"(a + 56u), "l"(b), "l"(b + 2u), "l"(b + 4u), "l"(b + 6u), "l"(b + BOX), "l"(b + BOX + 2u),
                   "l"(b + BOX + 4u), "l"(b + BOX + 6u), "r"(tc_idesc_bf16(N, false)), "r"(slot), "r"(sums), "r"(stage)
                 : "memory");
}

// A ring's position: the stage and how many times the ring has been round.
template <int STAGES>
struct GtRing {
    int stage = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == STAGES) {
            stage = 0;
            ++round;
        }
    }
};

template <int N>
__global__ void __launch_bounds__(GT_THREADS, 1)
w4a16_gate_up_tc_kernel(const GateUpTcParams p, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX)
{
    using L = GtSmem<N>;
    extern __shared__ __align__(1024) uint8_t gt_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(gt_smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(gt_smem + L::BARS);
    volatile int *flag = reinterpret_cast<volatile int *>(bars + L::COUNT);
    volatile uint32_t *slot_tm = reinterpret_cast<volatile uint32_t *>(flag + 1);
    auto bar = [&](int i) { return base + static_cast<uint32_t>(L::BARS + 8 * i); };
    const TcWait wait{flag, p.err};
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.err, 4);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::COUNT; ++i) {
            const bool warps4 = (i >= L::A_FULL && i < L::A_EMPTY) || i >= L::S_EMPTY;
            mbar_init(bar(i), i >= L::EMPTY && i < L::A_FULL ? 20 : i >= L::X_FULL ? 8 : warps4 ? 4 : 1);
        }
        *flag = 0;
        fence_barrier_init();
    }
    if (warp == GT_MMA_WARP) {
        tmem_alloc(smem_addr(const_cast<uint32_t *>(slot_tm)), GT_TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *slot_tm;
    pdl_launch_dependents();
    const int G = p.G, steps = (G + 1) / 2;     // stages of a tile
    const int mine = (p.tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);

    if (warp == GT_COPY_WARP) {
        const uint64_t once = policy_evict_first(), keep = policy_evict_last();
        const int total = mine * steps, ahead = min(total, L::STAGES);
        auto copy_w = [&](int i, int stage) {
            const int col0 = (static_cast<int>(blockIdx.x) + i / steps * static_cast<int>(gridDim.x)) * p.cols;
            const uint32_t st = base + stage * L::STAGE, fb = bar(L::FULL + stage);
            mbar_arrive_expect_tx(fb, static_cast<uint32_t>(2 * p.cols * 128 + 4 * N * 128));
            tma_load_2d(st, &tmW, i % steps * 32, col0, fb, once);
            tma_load_2d(st + GT_W_BYTES, &tmW, i % steps * 32, p.F + col0, fb, once);
        };
        auto copy_x = [&](int i, int stage) {
            const uint32_t st = base + stage * L::STAGE + L::X, fb = bar(L::FULL + stage);
#pragma unroll
            for (int j = 0; j < 4; ++j) tma_load_2d(st + j * N * 128, &tmX, i % steps * 256 + 64 * j, 0, fb, keep);
        };
        if (lane == 0)
            for (int i = 0; i < ahead; ++i) copy_w(i, i);
        pdl_wait_prior();                       // x may come from the kernel before
        if (lane == 0)
            for (int i = 0; i < ahead; ++i) copy_x(i, i);
        GtRing<L::STAGES> r;
        for (int i = ahead; i < total; ++i, r.next()) {
            wait(bar(L::EMPTY + r.stage), r.round);
            if (lane == 0) {
                copy_w(i, r.stage);
                copy_x(i, r.stage);
            }
            __syncwarp();
        }
    } else if (warp >= GT_MMA_WARP) {
        const int half = (warp - GT_MMA_WARP) >> 1, g = warp & 1;
        const uint32_t a0 = tmem + 256 * half, x0 = base + L::X + 2 * g * N * 128;
        const uint32_t a_full = bar(L::A_FULL + 2 * half + g), a_empty = bar(L::A_EMPTY + 2 * half + g);
        const uint32_t sums = bar(L::S_FULL + 4 * half + g), xs = bar(L::X_FULL + g);
        GtRing<L::STAGES> r;
        for (int i = 0; i < mine * steps; ++i, r.next()) {
            const int odd = i & 1;
            wait(xs + 16 * odd, i >> 1);
            if (i > 1) wait(sums + 16 * odd + 64, (i >> 1) - 1);
            wait(a_full, i);
            __syncwarp();
            tc_fence_after_sync();
            gt_products<N>(a0 + 128 + 64 * odd + 32 * g, a0 + 64 * g, desc_k_sw128(x0 + r.stage * L::STAGE), a_empty,
                           sums + 16 * odd, bar(L::EMPTY + r.stage));
        }
    } else if (warp < GT_SUM_WARP) {
        const int half = warp >> 3, g = (warp >> 2) & 1, row = threadIdx.x & (GT_ROWS - 1);
        const uint32_t a0 = tmem + 256 * half + 64 * g + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t a_full = bar(L::A_FULL + 2 * half + g), a_empty = bar(L::A_EMPTY + 2 * half + g);
        const uint32_t w = base + half * GT_W_BYTES + row * 128 + (((4 * g) ^ (row & 4)) << 4), swz = (row & 3) << 4;
        // the warp's eighth of the group's x
        const uint32_t x = base + L::X + 2 * g * N * 128 + (4 * half + (warp & 3)) * N * 32 + lane * 16;
        GtRing<L::STAGES> r;
        for (int i = 0; i < mine * steps; ++i, r.next()) {
            const uint32_t fb = bar(L::FULL + r.stage);
            wait(fb, r.round);
            uint4 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = lds128(w + r.stage * L::STAGE + ((j << 4) ^ swz));
#pragma unroll
            for (int u = 0; u < N / 16; ++u) {
                const uint32_t at = x + r.stage * L::STAGE + 512 * u;
                const uint4 v = lds128(at);
                sts128(at, make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                      __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)));
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(L::X_FULL + 2 * (i & 1) + g));
                mbar_arrive(fb + 8 * (L::EMPTY - L::FULL));
            }
            if (i > 0) wait(a_empty, i - 1);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[16];
                gt_levels(q[j].x, v);
                gt_levels(q[j].y, v + 4);
                gt_levels(q[j].z, v + 8);
                gt_levels(q[j].w, v + 12);
                tmem_st(a0 + 16 * j, v);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(a_full);
        }
    } else {
        const int half = (warp - GT_SUM_WARP) >> 2, row = threadIdx.x & (GT_ROWS - 1);
        const uint32_t d0 = tmem + 256 * half + 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t sums0 = bar(L::S_FULL + 4 * half);
        float *up = reinterpret_cast<float *>(gt_smem + L::UP) + row;
        uint32_t n = 0;                         // the block's stages so far
        for (int i = 0; i < mine; ++i) {
            const int col = (static_cast<int>(blockIdx.x) + i * static_cast<int>(gridDim.x)) * p.cols + row;
            const uint16_t *sc = p.scales + (static_cast<size_t>(half) * p.F + min(col, p.F - 1)) * G;
            float acc[N];
#pragma unroll
            for (int t = 0; t < N; ++t) acc[t] = 0.f;
            uint32_t s_next[GT_GROUPS] = {ldg_u16(sc), G > 1 ? ldg_u16(sc + 1) : 0u};   // read a stage ahead
            for (int k = 0; k < steps; ++k, ++n) {
                float s[GT_GROUPS];
#pragma unroll
                for (int g = 0; g < GT_GROUPS; ++g) {
                    s[g] = bf16_bits_to_float(s_next[g]);
                    const int grp = GT_GROUPS * (k + 1) + g;
                    s_next[g] = grp < G ? ldg_u16(sc + grp) : 0u;   // (a stage's absent group sums zeros)
                }
#pragma unroll
                for (int g = 0; g < GT_GROUPS; ++g) {
                    const int sum = 2 * (n & 1) + g;
                    wait(sums0 + 8 * sum, n >> 1);
                    __syncwarp();
                    tc_fence_after_sync();
#pragma unroll
                    for (int t0 = 0; t0 < N; t0 += 16) {
                        uint32_t d[16];
                        tmem_ld(d0 + 32 * sum + t0, d);
                        tmem_wait_ld();
                        if (t0 + 16 == N) {
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(sums0 + 8 * (8 + sum));
                        }
#pragma unroll
                        for (int t = 0; t < 16; ++t) acc[t0 + t] = fmaf(s[g], __uint_as_float(d[t]), acc[t0 + t]);
                    }
                }
            }
            if (i > 0) named_bar_sync(2, 2 * GT_ROWS);  // the tile before has been written
            if (half == 1)
#pragma unroll
                for (int t = 0; t < N; ++t) up[t * GT_ROWS] = GT_LEVEL_SCALE * acc[t];
            named_bar_sync(1, 2 * GT_ROWS);
            if (half == 0 && row < p.cols && col < p.F)
#pragma unroll
                for (int t = 0; t < N; ++t)
                    if (t < p.T)
                        p.h[static_cast<size_t>(t) * p.F + col] =
                            __bfloat16_as_ushort(__float2bfloat16_rn(gu_act(GT_LEVEL_SCALE * acc[t], p.act) * up[t * GT_ROWS]));
        }
    }
    // every copy has landed and every product is done: the warps above have
    // waited for each
    tc_fence_before_sync();
    __syncthreads();
    if (warp == GT_MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, GT_TMEM);
    }
}

}  // namespace sv
