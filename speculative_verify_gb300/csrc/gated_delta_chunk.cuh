// gated_delta_chunk.cuh -- the gated delta rule over whole prompts: blocks of
// 64 rows in closed form on the tensor cores.
//
// Within a block let G be the running sum of the log decays, r_k, r_q the
// inverse norms of keys and queries (1 without normalisation) and
//   A_ij = beta_i e^(G_i - G_j) r_k,i r_k,j (k_i . k_j)        i > j
//   M_ij = scale e^(G_i - G_j) r_q,i r_k,j (q_i . k_j)         i >= j
//   T    = (I + A)^-1 diag(beta).
// With the state S at the block's start the rows' updates and outputs are
//   r_i = v_i - e^(G_i) r_k,i (S k_i),     u = T r
//   o_i = scale e^(G_i) r_q,i (S q_i) + sum_j M_ij u_j
//   S'  = e^(G_n) S + sum_j u_j (e^(G_n - G_j) r_k,j k_j)^T.
//
// T, M and the row factors do not depend on the state, so a first kernel
// (delta_prep_kernel) computes them for all blocks and heads side by side; a
// second (delta_scan_kernel) walks the blocks of one head of one sequence
// with the state in registers.
//
// Precision.  Keys and queries enter the bf16 tensor-core products as they
// come, their norms staying outside as fp32 factors.  The fp32 factors --
// state, T, M, r, u -- enter as two bf16 terms each (16 bits; of a product of
// two such factors the lo x lo part is left out).  The state then comes out
// within 5e-6 of the rule in exact arithmetic (row by row in fp32: 2e-7), well
// below the 2^-9 of the bf16 rows that it is made from and of the outputs.
//
// Measured, 16 key and 48 value heads of 128: 4 prompts of 8,192 rows 747 us
// (prep 275), one of 3,847 rows 215 (42), nine ragged ones with 6,317 rows 190.
// Prep is bound by its instructions (4,700 a warp, 43 % issue), the scan by
// the chain of a block.
#pragma once

#include <cuda.h>

#include "gated_delta.cuh"
#include "tc_ops.cuh"
#include "w4a16_stream.cuh"

namespace sv {

constexpr int DC_ROWS = 64;                     // rows of a block
constexpr int DC_MAT = DC_ROWS * 128;           // bytes of one 64 x 64 bf16 matrix, 128-byte swizzled
constexpr int DC_FACTORS = 1024;                // bytes of a block's row factors
constexpr int DC_BLOCK = 4 * DC_MAT + DC_FACTORS;   // T transposed (two terms), M (two terms), factors
constexpr int DC_FLAGS = 4096;                  // bytes of hand-over flags before the blocks, one word a CTA

struct DeltaChunkParams {
    DeltaParams d;                              // rows, shape, state; T and prev unused
    const int32_t *cu;                          // [B + 1] first rows
    int R, B;                                   // rows in all, sequences
    int zero_init;
    unsigned *flags;                            // [DC_FLAGS / 4], zero when the scan starts
    uint8_t *blocks;                            // [R / 64 + B][Hv][DC_BLOCK]
    int32_t *cu_run;                            // [B + 1]: cu as the scan reads it
};

// The rows of sequence b: cu[b] .. cu[b + 1], kept within [0, R].
__device__ __forceinline__ void gd_range(const int32_t *cu, int R, int b, int &begin, int &end)
{
    begin = min(max(cu[b], 0), R);
    end = min(max(cu[b + 1], begin), R);
}

// A sequence's first block in the workspace.  Blocks of a sequence are
// numbered one after another, and floor(begin / 64) + b leaves room for the
// part block of every sequence before it.
__device__ __forceinline__ int dc_base(int begin, int b) { return begin / DC_ROWS + b; }

// Row by row, for short sequences.  Grid: x = dv / GD_COLS, y = Hv, z = B.
template <int DK>
__global__ void __launch_bounds__(GD_THREADS, gd_blocks(DK)) gated_delta_rows_kernel(const DeltaChunkParams cp)
{
    extern __shared__ __align__(16) float gd_smem[];
    const DeltaParams &p = cp.d;
    const int col0 = blockIdx.x * GD_COLS, hv = blockIdx.y, b = blockIdx.z;
    const int i = threadIdx.x & 3, col = threadIdx.x >> 2;
    const GdSmem<DK> sm(gd_smem, GD_MAX_ROWS);
    pdl_launch_dependents();
    pdl_wait_prior();
    int begin, end;
    gd_range(cp.cu, cp.R, b, begin, end);
    const int slot = gd_slot(p.state_idx, p.n_slots, b, p.err);
    uint16_t *o = p.o + begin * p.ldo + static_cast<long long>(hv) * p.dv + col0;
    if (slot < 0) {
        for (int t = begin; t < end; ++t, o += p.ldo)
            if (i == 0) o[col] = 0;
        return;
    }
    float *s = p.state + ((static_cast<long long>(slot) * p.Hv + hv) * p.dv + col0 + col) * DK;
    GdState<DK> st;
    if (cp.zero_init)
        st.zero();
    else
        st.load(s, i);
    for (int r0 = begin; r0 < end; r0 += GD_MAX_ROWS) {
        const int n = min(GD_MAX_ROWS, end - r0);
        GdFirst<DK> f;
        gd_first<DK>(p, p.rows, r0, n, hv, col0, true, f);
        const bool running = gd_stage<DK>(p, p.rows, r0, n, hv, col0, sm, true, f);
        gd_rows<DK, true>(st, sm, n, running, o, p.ldo);
        o += n * p.ldo;
        __syncthreads();
    }
    st.store(s, i);
}

// ----------------------------------------------------------------- prep
//
// One CTA per block of rows and key head: K K^T and Q K^T once, then T and M
// of each value head.  A warp has 16 rows (row block w) of both products and
// keeps them in registers for all value heads.
//
// Decays: e^(G_i - G_j) below the diagonal blocks is e^(G_i - G_r) e^(G_r -
// G_j) with r the first row of i's block, both at most 1 for decays; within a
// diagonal block it is taken directly.  Exponentials are the fast ones: their
// error, 2^-22 and 2^-24 of the exponent, is within the operands' 16 bits.
//
// T: the 16 x 16 diagonal blocks of (I + A)^-1 by forward substitution (fp32,
// a column a lane), the others by T_IJ = -T_II sum_K A_IK T_KJ on the tensor
// cores.  They are computed transposed, T_IJ^T = -(sum_K T_KJ^T A_IK^T) T_II^T:
// an accumulator's registers are then the next product's A operand as they
// stand, and warp J can do all of column block J.  Operands in two bf16 terms.
// T diag(beta) is stored transposed, [j][i], which pairs the columns that a
// lane has.

// Byte of element (row, column) of a 64 x 64 bf16 matrix whose 128-byte rows
// are swizzled in 16-byte pieces, as the tensor cores' descriptors expect.
__device__ __forceinline__ int dc_swizzled(int row, int col)
{
    return row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}

constexpr int DC_HEADS = 4;                     // value heads whose gates are staged at once, one a warp
constexpr int DC_AST = DC_ROWS + 8;             // columns of a row of A in shared memory
constexpr int DC_TST = 24;                      // columns of a row of a diagonal block

template <int DK>
struct DcPrepSmem {
    union {
        struct {
            uint16_t k[DC_ROWS][DK + 8], q[DC_ROWS][DK + 8];
        } in;
        struct {
            uint16_t a_hi[DC_ROWS][DC_AST], a_lo[DC_ROWS][DC_AST];  // below the diagonal blocks
            uint16_t t_hi[4][16][DC_TST], t_lo[4][16][DC_TST];      // diagonal blocks of (I + A)^-1
            float d[4][16][20];                                     // diagonal blocks of A
        } w;
    } u;
    float rk[DC_ROWS], rq[DC_ROWS];
    float beta[DC_HEADS][DC_ROWS], g_hi[DC_HEADS][DC_ROWS], g_lo[DC_HEADS][DC_ROWS];
    float near[DC_HEADS][DC_ROWS];              // e^(G_i - G_r)
    float far[DC_HEADS][4][DC_ROWS];            // [row block][j]: e^(G_r - G_j)
    int seq;
    unsigned long long claimed;                 // blocks of all sequences
};

// d (two n8 tiles of 16 rows) += a x b over 16 columns, both in two terms.
__device__ __forceinline__ void mma_split(float (&d)[2][4], const uint32_t (&a_hi)[4], const uint32_t (&a_lo)[4],
                                          const uint32_t (&b_hi)[4], const uint32_t (&b_lo)[4])
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        mma_bf16_16816(d[j], a_lo[0], a_lo[1], a_lo[2], a_lo[3], b_hi[2 * j], b_hi[2 * j + 1]);
        mma_bf16_16816(d[j], a_hi[0], a_hi[1], a_hi[2], a_hi[3], b_lo[2 * j], b_lo[2 * j + 1]);
        mma_bf16_16816(d[j], a_hi[0], a_hi[1], a_hi[2], a_hi[3], b_hi[2 * j], b_hi[2 * j + 1]);
    }
}

// Grid: x = R / 64 + B blocks, y = Hk; 128 threads.
template <int DK>
__global__ void __launch_bounds__(128, 4) delta_prep_kernel(const DeltaChunkParams cp)
{
    extern __shared__ __align__(16) uint8_t dc_smem[];
    DcPrepSmem<DK> &sm = *reinterpret_cast<DcPrepSmem<DK> *>(dc_smem);
    const DeltaParams &p = cp.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int id = blockIdx.x, hk = blockIdx.y, rep = p.Hv / p.Hk;
    pdl_launch_dependents();
    pdl_wait_prior();
    if (id == 0 && hk == 0) {
        for (int i = tid; i < DC_FLAGS / 4; i += 128) cp.flags[i] = 0u;
        // The scan counts blocks in 32 bits.  Rows claimed twice (by cu_seqlens
        // that decrease) may be any number of them: with more than the rows have
        // once, the sequences count as empty.
        if (tid == 0) sm.claimed = 0;
        __syncthreads();
        unsigned long long mine = 0;
        for (int b = tid; b < cp.B; b += 128) {
            int begin, end;
            gd_range(cp.cu, cp.R, b, begin, end);
            mine += static_cast<unsigned>(end - begin + DC_ROWS - 1) / DC_ROWS;
        }
        atomicAdd(&sm.claimed, mine);
        __syncthreads();
        const bool bad = sm.claimed > static_cast<unsigned>(cp.R / DC_ROWS + cp.B);
        if (bad && tid == 0) atomicOr(p.err, 16);       // SV_DEVERR_BAD_SEQLENS
        for (int b = tid; b <= cp.B; b += 128) cp.cu_run[b] = bad ? 0 : cp.cu[b];
    }
    // the sequence whose blocks hold this one (the last such, where rows are
    // claimed twice, which cu_seqlens must not do)
    if (tid == 0) sm.seq = -1;
    __syncthreads();
    for (int b = tid; b < cp.B; b += 128) {
        int begin, end;
        gd_range(cp.cu, cp.R, b, begin, end);
        const int base = dc_base(begin, b);
        if (id >= base && id < base + (end - begin + DC_ROWS - 1) / DC_ROWS) atomicMax(&sm.seq, b);
    }
    __syncthreads();
    const int seq = sm.seq;
    if (seq < 0) return;                        // a spare number
    int begin, end;
    gd_range(cp.cu, cp.R, seq, begin, end);
    const int row0 = begin + (id - dc_base(begin, seq)) * DC_ROWS;
    const int n = min(DC_ROWS, end - row0);

    // keys and queries; rows past the sequence's end are zero
    constexpr int PR = DK / 8;                  // 16-byte pieces of a row
    {
        constexpr int PT = DC_ROWS * PR / 128;  // pieces of a thread
        uint4 kv[PT], qv[PT];
#pragma unroll
        for (int u = 0; u < PT; ++u) {
            const int i = tid + u * 128, t = i / PR, j = (i % PR) * 8;
            kv[u] = qv[u] = make_uint4(0u, 0u, 0u, 0u);
            if (t < n) {
                kv[u] = __ldg(reinterpret_cast<const uint4 *>(p.rows.k + (row0 + t) * p.rows.ldk + hk * DK + j));
                qv[u] = __ldg(reinterpret_cast<const uint4 *>(p.rows.q + (row0 + t) * p.rows.ldq + hk * DK + j));
            }
        }
#pragma unroll
        for (int u = 0; u < PT; ++u) {
            const int i = tid + u * 128, t = i / PR, j = (i % PR) * 8;
            *reinterpret_cast<uint4 *>(&sm.u.in.k[t][j]) = kv[u];
            *reinterpret_cast<uint4 *>(&sm.u.in.q[t][j]) = qv[u];
        }
    }
    __syncthreads();
    // k_i . k_j and q_i . k_j for the warp's rows i and j up to their block;
    // q_i . q_i from the diagonal of the block's q q^T
    float ck[8][4], cq[8][4], qq[2][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ck[j][e] = cq[j][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) qq[j][e] = 0.f;
    const uint32_t arow = static_cast<uint32_t>(((warp * 16 + (lane & 15)) * (DK + 8) + (lane >> 4) * 8) * 2);
    const uint32_t brow = static_cast<uint32_t>((((lane & 7) + ((lane >> 4) << 3)) * (DK + 8) + ((lane >> 3) & 1) * 8) * 2);
    {
        const uint32_t k0 = smem_addr(&sm.u.in.k[0][0]), q0 = smem_addr(&sm.u.in.q[0][0]);
#pragma unroll
        for (int s = 0; s < DK / 16; ++s) {
            uint32_t ak[4], aq[4], b[4];
            ldmatrix_x4(ak, k0 + arow + 32u * s);
            ldmatrix_x4(aq, q0 + arow + 32u * s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > warp) break;
                ldmatrix_x4(b, k0 + brow + static_cast<uint32_t>(j * 16 * (DK + 8) * 2) + 32u * s);
                mma_bf16_16816(ck[2 * j], ak[0], ak[1], ak[2], ak[3], b[0], b[1]);
                mma_bf16_16816(ck[2 * j + 1], ak[0], ak[1], ak[2], ak[3], b[2], b[3]);
                mma_bf16_16816(cq[2 * j], aq[0], aq[1], aq[2], aq[3], b[0], b[1]);
                mma_bf16_16816(cq[2 * j + 1], aq[0], aq[1], aq[2], aq[3], b[2], b[3]);
            }
            // rows as columns: tile j of the block is rows 8 j .. of it
            mma_bf16_16816(qq[0], aq[0], aq[1], aq[2], aq[3], aq[0], aq[2]);
            mma_bf16_16816(qq[1], aq[0], aq[1], aq[2], aq[3], aq[1], aq[3]);
        }
    }
    // the diagonal: row g of tile 0 and row g + 8 of tile 1, columns 2c, 2c + 1
    if ((g >> 1) == c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float kk = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j == warp) kk = (g & 1) ? ck[2 * j + h][2 * h + 1] : ck[2 * j + h][2 * h];
            const float q2 = (g & 1) ? qq[h][2 * h + 1] : qq[h][2 * h];
            const int i = warp * 16 + g + 8 * h;
            sm.rk[i] = p.l2norm ? 1.f / sqrtf(kk + GD_L2_EPS) : 1.f;
            sm.rq[i] = p.scale * (p.l2norm ? 1.f / sqrtf(q2 + GD_L2_EPS) : 1.f);
        }
    }
    uint8_t *blocks = cp.blocks + (static_cast<size_t>(id) * p.Hv + hk * rep) * DC_BLOCK;
    const uint32_t a_hi0 = smem_addr(&sm.u.w.a_hi[0][0]), a_lo0 = smem_addr(&sm.u.w.a_lo[0][0]);
    const uint32_t t_hi0 = smem_addr(&sm.u.w.t_hi[0][0][0]), t_lo0 = smem_addr(&sm.u.w.t_lo[0][0][0]);
    // a lane's row of ldmatrix: plain (B operand, two n8 tiles) and transposed (A operand)
    const int b_r = (lane & 7) + ((lane >> 4) << 3), b_c = ((lane >> 3) & 1) * 8;
    for (int r = 0; r < rep; ++r) {
        __syncthreads();                        // the inputs, or the last head's matrices, have been read
        const int e4 = r & (DC_HEADS - 1);
        if (e4 == 0) {
            // gates of the next heads, one a warp, two rows a lane
            const int hv = hk * rep + r + warp;
            if (r + warp < rep) {
                Sum2 G[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    float v = t < n ? p.rows.g[(row0 + t) * p.rows.ldg + hv] : 0.f;
                    if (v < GD_MIN_LOG) v = GD_MIN_LOG;
                    G[e] = Sum2{v, 0.f};
                    sm.beta[warp][t] = t < n ? p.rows.beta[(row0 + t) * p.rows.ldg + hv] : 0.f;
                }
                Sum2 run = add2(G[0], G[1]);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const Sum2 below{__shfl_up_sync(0xFFFFFFFFu, run.hi, o), __shfl_up_sync(0xFFFFFFFFu, run.lo, o)};
                    if (lane >= o) run = add2(below, run);
                }
                Sum2 before{__shfl_up_sync(0xFFFFFFFFu, run.hi, 1), __shfl_up_sync(0xFFFFFFFFu, run.lo, 1)};
                if (lane == 0) before = Sum2{0.f, 0.f};
                G[0] = add2(before, G[0]);
                G[1] = run;
                const float hi[2] = {G[0].hi, G[1].hi}, lo[2] = {G[0].lo, G[1].lo};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sm.g_hi[warp][2 * lane + e] = hi[e];
                    sm.g_lo[warp][2 * lane + e] = lo[e];
                }
                const float end_hi = __shfl_sync(0xFFFFFFFFu, hi[1], 31), end_lo = __shfl_sync(0xFFFFFFFFu, lo[1], 31);
                float *f = reinterpret_cast<float *>(blocks + static_cast<size_t>(r + warp) * DC_BLOCK + 4 * DC_MAT);
                float fe[2], fl[2], fq[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // row factors: -e^G r_k, e^(G_n - G) r_k, scale e^G r_q
                    const int t = 2 * lane + e;
                    const float eg = __expf(hi[e] + lo[e]);
                    fe[e] = t < n ? -eg * sm.rk[t] : 0.f;
                    fl[e] = t < n ? __expf((end_hi - hi[e]) + (end_lo - lo[e])) * sm.rk[t] : 0.f;
                    fq[e] = t < n ? eg * sm.rq[t] : 0.f;
                    const int own_block = t >> 4;
#pragma unroll
                    for (int I = 0; I < 4; ++I) {
                        const float ref_hi = __shfl_sync(0xFFFFFFFFu, hi[0], 8 * I), ref_lo = __shfl_sync(0xFFFFFFFFu, lo[0], 8 * I);
                        if (I == own_block) sm.near[warp][t] = __expf((hi[e] - ref_hi) + (lo[e] - ref_lo));
                        if (I > own_block) sm.far[warp][I][t] = __expf((ref_hi - hi[e]) + (ref_lo - lo[e])) * sm.rk[t];
                    }
                }
                *reinterpret_cast<float2 *>(f + 2 * lane) = make_float2(fe[0], fe[1]);
                *reinterpret_cast<float2 *>(f + DC_ROWS + 2 * lane) = make_float2(fl[0], fl[1]);
                *reinterpret_cast<float2 *>(f + 2 * DC_ROWS + 2 * lane) = make_float2(fq[0], fq[1]);
                if (lane == 0) f[3 * DC_ROWS] = __expf(end_hi + end_lo);
            }
            __syncthreads();
        }
        uint8_t *out = blocks + static_cast<size_t>(r) * DC_BLOCK;
        // M, and A: its diagonal blocks in fp32, the rest in two terms
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int il = g + 8 * h, i = warp * 16 + il;
            const float bi = i < n ? sm.beta[e4][i] * sm.rk[i] : 0.f, qi = i < n ? sm.rq[i] : 0.f;
            const float near = sm.near[e4][i], bn = bi * near, qn = qi * near;
            const float gi = sm.g_hi[e4][i], gl = sm.g_lo[e4][i];
#pragma unroll
            for (int j8 = 0; j8 < 8; ++j8) {
                if ((j8 >> 1) > warp) break;
                const int j0 = j8 * 8 + c * 2;
                float m[2], a[2];
                if ((j8 >> 1) < warp) {
                    const float2 far = *reinterpret_cast<const float2 *>(&sm.far[e4][warp][j0]);
                    m[0] = cq[j8][2 * h] * (far.x * qn);
                    m[1] = cq[j8][2 * h + 1] * (far.y * qn);
                    a[0] = ck[j8][2 * h] * (far.x * bn);
                    a[1] = ck[j8][2 * h + 1] * (far.y * bn);
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = j0 + e;
                        const float d = j <= i ? __expf((gi - sm.g_hi[e4][j]) + (gl - sm.g_lo[e4][j])) * sm.rk[j] : 0.f;
                        m[e] = j <= i ? cq[j8][2 * h + e] * (d * qi) : 0.f;
                        a[e] = j < i ? ck[j8][2 * h + e] * (d * bi) : 0.f;
                    }
                }
                uint32_t hi, lo;
                split_bf16x2(m[0], m[1], hi, lo);
                *reinterpret_cast<uint32_t *>(out + 2 * DC_MAT + dc_swizzled(i, j0)) = hi;
                *reinterpret_cast<uint32_t *>(out + 3 * DC_MAT + dc_swizzled(i, j0)) = lo;
                if ((j8 >> 1) < warp) {
                    split_bf16x2(a[0], a[1], hi, lo);
                    *reinterpret_cast<uint32_t *>(&sm.u.w.a_hi[i][j0]) = hi;
                    *reinterpret_cast<uint32_t *>(&sm.u.w.a_lo[i][j0]) = lo;
                } else {
                    *reinterpret_cast<float2 *>(&sm.u.w.d[warp][il][j0 & 15]) = make_float2(a[0], a[1]);
                }
            }
        }
        __syncwarp();
        if (lane < 16) {
            // column `lane` of the warp's diagonal block of (I + A)^-1
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(&sm.u.w.d[warp][i][m]);
                    s0 = fmaf(-a.x, t[m], s0);
                    if (m + 1 < i) s1 = fmaf(-a.y, t[m + 1], s1);
                    if (m + 2 < i) s0 = fmaf(-a.z, t[m + 2], s0);
                    if (m + 3 < i) s1 = fmaf(-a.w, t[m + 3], s1);
                }
                t[i] = s0 + s1;
            }
            const float b = sm.beta[e4][warp * 16 + lane];
            uint32_t oh[8], ol[8];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                uint32_t hi, lo;
                split_bf16x2(t[i], t[i + 1], hi, lo);
                sm.u.w.t_hi[warp][i][lane] = static_cast<uint16_t>(hi);
                sm.u.w.t_hi[warp][i + 1][lane] = static_cast<uint16_t>(hi >> 16);
                sm.u.w.t_lo[warp][i][lane] = static_cast<uint16_t>(lo);
                sm.u.w.t_lo[warp][i + 1][lane] = static_cast<uint16_t>(lo >> 16);
                split_bf16x2(t[i] * b, t[i + 1] * b, oh[i / 2], ol[i / 2]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = dc_swizzled(warp * 16 + lane, warp * 16 + 8 * e);
                *reinterpret_cast<uint4 *>(out + at) = make_uint4(oh[4 * e], oh[4 * e + 1], oh[4 * e + 2], oh[4 * e + 3]);
                *reinterpret_cast<uint4 *>(out + DC_MAT + at) = make_uint4(ol[4 * e], ol[4 * e + 1], ol[4 * e + 2], ol[4 * e + 3]);
            }
        }
        __syncthreads();
        if (warp < 3) {
            // column block J = warp of T below its diagonal block, transposed
            const int J = warp;
            uint32_t th[4][4], tl[4][4];        // [row block K]: T_KJ^T as an A operand
            {
                const uint32_t at = static_cast<uint32_t>(((J * 16 + (lane & 7) + ((lane >> 4) << 3)) * DC_TST + ((lane >> 3) & 1) * 8) * 2);
                ldmatrix_x4_trans(th[0], t_hi0 + at);
                ldmatrix_x4_trans(tl[0], t_lo0 + at);
            }
#pragma unroll
            for (int d = 1; d < 4; ++d) {       // row block I = J + d
                const int I = J + d;
                if (I > 3) break;
                float x[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j][e] = 0.f;
                uint32_t bh[4], bl[4];
#pragma unroll
                for (int k = 0; k < d; ++k) {   // K = J + k
                    const uint32_t at = static_cast<uint32_t>(((16 * I + b_r) * DC_AST + 16 * (J + k) + b_c) * 2);
                    ldmatrix_x4(bh, a_hi0 + at);
                    ldmatrix_x4(bl, a_lo0 + at);
                    mma_split(x, th[k], tl[k], bh, bl);
                }
                uint32_t xh[4], xl[4];
                split_bf16x2(-x[0][0], -x[0][1], xh[0], xl[0]);
                split_bf16x2(-x[0][2], -x[0][3], xh[1], xl[1]);
                split_bf16x2(-x[1][0], -x[1][1], xh[2], xl[2]);
                split_bf16x2(-x[1][2], -x[1][3], xh[3], xl[3]);
                const uint32_t at = static_cast<uint32_t>(((I * 16 + b_r) * DC_TST + b_c) * 2);
                ldmatrix_x4(bh, t_hi0 + at);
                ldmatrix_x4(bl, t_lo0 + at);
                float y[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[j][e] = 0.f;
                mma_split(y, xh, xl, bh, bl);
                if (d < 3) {
                    split_bf16x2(y[0][0], y[0][1], th[d][0], tl[d][0]);
                    split_bf16x2(y[0][2], y[0][3], th[d][1], tl[d][1]);
                    split_bf16x2(y[1][0], y[1][1], th[d][2], tl[d][2]);
                    split_bf16x2(y[1][2], y[1][3], th[d][3], tl[d][3]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j = 16 * J + g + 8 * h;
                    const float b = sm.beta[e4][j];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        uint32_t hi, lo;
                        split_bf16x2(y[t][2 * h] * b, y[t][2 * h + 1] * b, hi, lo);
                        const int o = dc_swizzled(j, 16 * I + 8 * t + 2 * c);
                        *reinterpret_cast<uint32_t *>(out + o) = hi;
                        *reinterpret_cast<uint32_t *>(out + DC_MAT + o) = lo;
                    }
                }
            }
        }
    }
}

// ----------------------------------------------------------------- scan
//
// Everything is transposed, with the value dimension on the tensor memory's
// lanes (state row l on lane l), so that the state, r and u are A operands in
// tensor memory and the keys, queries, T and M are B operands in shared
// memory exactly as they are loaded.  Tensor memory, in columns:
//
//   phase  product                               accumulator
//   P      S (2 terms, 0..127) x K               P  128..191
//   O      S x Q                                 O  320..383
//   U      r (2, 192..255) x T (2)               U  256..319
//   D      u' (2, 448..511) x K                  D  128..255 (over P and r)
//   M      u (2, 256..319 over U) x M (2)        M  384..447
//
// (of a product of two two-term factors lo x lo is left out).  Warps 0-15
// convert between the products: warp w has lanes 32 (w & 3) .. + 31 and a
// quarter w >> 2 of the columns; the state's fp32 values stay in their
// registers; they write a block's outputs while the next one's P runs.  Warp
// 16 issues the products, warp 17 the loads, two blocks ahead.
//
// The chain of a block, P, r, U, u', D, S, bounds the kernel; O, M and the
// outputs fill its gaps.  D goes by halves of the state's columns: the first
// half's new state is converted, and P's steps over it begun, while the second
// half's D and conversion run (4 prompts of 8,192 rows 764 -> 745 us).  A block
// of 128 x 128 states then takes 5,400 cycles; by clock stamps before that, of
// 5,700, P 1,100 with its hand-offs, r 550, U 650, u' 700, D 900, S 950, the
// rest outputs and values.  A 128 x 64 x 16 product with its A operand in
// tensor memory takes up to 56 cycles, so O is issued in two halves, into the
// gaps after P and after U, where it delays neither.

// Work.  The chains of all heads and sequences are laid end to end, each as
// long as its blocks and DS_EXTRA more for its start and end (loading and
// storing a state costs about two blocks' time), and cut into equal parts, at
// least as long as the longest chain, one for each CTA.
// A chain that a cut divides has its first blocks at the start of the later
// CTA's part -- which runs them at once -- and its last ones at the end of
// the earlier CTA's, which takes the state over when it gets there: with 192
// chains of equal length on 152 SMs the whole takes 1.26 chains' time, not
// two.  A CTA waits for CTAs of lower blockIdx only.

constexpr int DS_WARPS = 16;                    // converting warps
constexpr int DS_MMA = 16, DS_LOAD = 17;        // the issuing warps
constexpr int DS_THREADS = 18 * 32;
constexpr int DS_EXTRA = 2;
constexpr uint32_t DS_COLS = 512;
constexpr uint32_t DS_SHI = 0, DS_SLO = 64, DS_P = 128, DS_R = 192, DS_U = 256, DS_O = 320, DS_M = 384, DS_UP = 448;

template <int DK>
struct DsSmem {                                 // from a 1024-byte boundary
    static constexpr int TILE = DC_ROWS * DK * 2;   // keys or queries: DK / 64 boxes of [64 rows][128 bytes]
    static constexpr int K = 0, Q = TILE, MATS = 2 * TILE, V = MATS + 4 * DC_MAT;   // V [64][dv]
    static constexpr int STAGE = V + DC_ROWS * 128 * 2;
    static constexpr int F = 2 * STAGE;         // row factors, four buffers: they are read later than the rest
    static constexpr int BARS = F + 4 * DC_FACTORS;
    static constexpr int BYTES = BARS + 256;
};

// Barriers that a waiter could find two phases ahead come in pairs, one for
// even and one for odd steps: their next phase needs the waiter to go on.
enum { B_FULL0, B_FULL1, B_P, B_U, B_D0, B_D1, B_M0, B_M1, B_SREADY0, B_SREADY1, B_RREADY, B_UREADY, B_MREADY, B_YFREE, B_COUNT };

// A CTA's part of the chains: segments of one head of one sequence each.
struct DsWalk {
    const DeltaChunkParams *cp;
    int pos, stop, lo;                          // next place, end and start of the part
    int b, first, length;                       // the sequence of `pos`, its first place, the length of its chains
    // the current segment: blocks c0 .. c1 - 1 of head hv of sequence b
    int begin, end, blocks, slot, hv, c0, c1;
    bool takes, gives;                          // another CTA ran the blocks before, runs those after

    __device__ __forceinline__ int blocks_of(int s, int &bg, int &en, int &sl) const
    {
        gd_range(cp->cu, cp->R, s, bg, en);
        sl = cp->d.state_idx ? cp->d.state_idx[s] : s;
        return sl < 0 || sl >= cp->d.n_slots ? 0 : (en - bg + DC_ROWS - 1) / DC_ROWS;
    }
    // Places of sequence s's chains.
    __device__ __forceinline__ int places_of(int s) const
    {
        int bg, en, sl;
        const int nb = blocks_of(s, bg, en, sl);
        return nb ? (nb + DS_EXTRA) * cp->d.Hv : 0;
    }
    // Part k of `parts` (whole warps call it).
    __device__ __forceinline__ void start(const DeltaChunkParams *c, int k, int parts)
    {
        cp = c;
        const int lane = threadIdx.x & 31;
        int total = 0, most = 0;
        for (int s = lane; s < cp->B; s += 32) {
            const int n = places_of(s);
            total += n;
            most = max(most, n);
        }
        total = __reduce_add_sync(0xFFFFFFFFu, total);
        most = __reduce_max_sync(0xFFFFFFFFu, most) / cp->d.Hv;
        const int cap = max(most, (total + parts - 1) / parts);
        // (k cap may be far past the end)
        lo = static_cast<int>(min(static_cast<long long>(k) * cap, static_cast<long long>(total)));
        stop = min(total, lo + cap);
        pos = lo;
        b = first = 0;
        for (int s0 = 0; s0 < cp->B && lo < stop; s0 += 32) {
            const int s = s0 + lane, mine = s < cp->B ? places_of(s) : 0;
            int run = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int below = __shfl_up_sync(0xFFFFFFFFu, run, o);
                if (lane >= o) run += below;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, first + run > pos);
            if (past) {
                const int w = __ffs(past) - 1;
                b = s0 + w;
                first += __shfl_sync(0xFFFFFFFFu, run - mine, w);
                break;
            }
            first += __shfl_sync(0xFFFFFFFFu, run, 31);
        }
        length = 0;
    }
    // The next segment that has blocks; false at the part's end.
    __device__ __forceinline__ bool next()
    {
        while (pos < stop) {
            while (length == 0 || length * cp->d.Hv <= pos - first) {
                // the sequence of `pos`: this one (not looked at yet) or a later one
                if (length) {
                    first += length * cp->d.Hv;
                    ++b;
                }
                while ((blocks = blocks_of(b, begin, end, slot)) == 0) ++b;
                length = blocks + DS_EXTRA;
            }
            hv = (pos - first) / length;
            const int s = first + hv * length, e = s + length;
            // of a chain with L places after the cut, the later part's CTA has the first L - 1 blocks
            c0 = e > stop ? e - stop - 1 : 0;
            c1 = pos > s ? e - pos - 1 : blocks;
            takes = c0 > 0;                     // the CTA of the part after has the first c0 blocks
            gives = c1 < blocks;                // (pos == lo) the CTA of the part before has the rest
            pos = min(e, stop);
            if (c0 < c1) return true;
        }
        return false;
    }
};

template <int DK>
__global__ void __launch_bounds__(DS_THREADS, 1)
delta_scan_kernel(const __grid_constant__ DeltaChunkParams cp, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmV)
{
    extern __shared__ __align__(1024) uint8_t ds_smem[];
    using L = DsSmem<DK>;
    constexpr int HALVES = DK / 64;             // D, and P's steps, go by 64 state columns
    const DeltaParams &p = cp.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = gridDim.x - 1 - blockIdx.x;
    const uint32_t base = smem_addr(ds_smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ds_smem + L::BARS);
    volatile int *flag = reinterpret_cast<volatile int *>(bars + B_COUNT);
    volatile uint32_t *slot_tm = reinterpret_cast<volatile uint32_t *>(flag + 1);
    auto bar = [&](int i) { return base + static_cast<uint32_t>(L::BARS + 8 * i); };
    const TcWait wait{flag, p.err};

    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.err, 4);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), i < B_SREADY0 ? 1 : i < B_RREADY ? DS_WARPS / HALVES : DS_WARPS);
        *flag = 0;
        fence_barrier_init();
    }
    if (warp == DS_MMA) {
        tmem_alloc(smem_addr(const_cast<uint32_t *>(slot_tm)), DS_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *slot_tm;
    pdl_launch_dependents();
    pdl_wait_prior();
    DsWalk w;
    w.start(&cp, part, gridDim.x);

    if (warp == DS_LOAD) {
        // ------------------------------------------------ loads, step t into stage t & 1
        const uint64_t keep = policy_evict_last(), once = policy_evict_first();
        uint32_t t = 0;
        while (w.next())
            for (int c = w.c0; c < w.c1; ++c, ++t) {
                // Step t - 2's products are done, so its values have been read
                // (r came before U), and so have the row factors of step
                // t - 4 (step t - 2's O followed the outputs of step t - 3).
                if (t > 1) wait(bar(B_M0 + (t & 1)), (t >> 1) - 1);
                if (lane == 0) {
                    const uint32_t st = base + (t & 1) * L::STAGE, fb = bar(B_FULL0 + (t & 1));
                    const int row = w.begin + c * DC_ROWS, hk = w.hv / (p.Hv / p.Hk);
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(2 * L::TILE + DC_BLOCK + DC_ROWS * p.dv * 2));
#pragma unroll
                    for (int j = 0; j < DK / 64; ++j)
                        tma_load_2d(st + L::K + j * DC_ROWS * 128, &tmK, hk * DK + 64 * j, row, fb, keep);
                    tma_load_2d(st + L::V, &tmV, w.hv * p.dv, row, fb, once);
                    const uint8_t *blk = cp.blocks + (static_cast<size_t>(dc_base(w.begin, w.b) + c) * p.Hv + w.hv) * DC_BLOCK;
                    bulk_g2s(st + L::MATS, blk, 4 * DC_MAT, fb, once);
                    bulk_g2s(base + L::F + (t & 3) * DC_FACTORS, blk + 4 * DC_MAT, DC_FACTORS, fb, once);
#pragma unroll
                    for (int j = 0; j < DK / 64; ++j)
                        tma_load_2d(st + L::Q + j * DC_ROWS * 128, &tmQ, hk * DK + 64 * j, row, fb, keep);
                    if (c + 1 < w.c1) {         // the next block's on its way to L2
#pragma unroll
                        for (int j = 0; j < DK / 64; ++j) {
                            prefetch_l2_2d(&tmK, hk * DK + 64 * j, row + DC_ROWS);
                            prefetch_l2_2d(&tmQ, hk * DK + 64 * j, row + DC_ROWS);
                        }
                        prefetch_l2_2d(&tmV, w.hv * p.dv, row + DC_ROWS);
                        prefetch_l2(blk + static_cast<size_t>(p.Hv) * DC_BLOCK, DC_BLOCK);
                    }
                }
                __syncwarp();
            }
    } else if (warp == DS_MMA) {
        // ------------------------------------------------ products
        uint32_t t = 0;
        while (w.next())
            for (int c = w.c0; c < w.c1; ++c, ++t) {
                const uint32_t st = base + (t & 1) * L::STAGE, kb = st + L::K, qb = st + L::Q, mb = st + L::MATS;
                const uint32_t y = tmem + DS_O;
                auto s_product = [&](uint32_t d, uint32_t rows, int s) {
                    const uint64_t b = desc_k_sw128(rows + (s >> 2) * DC_ROWS * 128 + (s & 3) * 32);
                    tc_mma_f16_ts_warp(d, tmem + DS_SHI + 8 * s, b, tc_idesc_bf16(64, false), s > 0);
                    tc_mma_f16_ts_warp(d, tmem + DS_SLO + 8 * s, b, tc_idesc_bf16(64, false), 1);
                };
                // P: S x K
                wait(bar(B_FULL0 + (t & 1)), t >> 1);
#pragma unroll
                for (int half = 0; half < HALVES; ++half) {
                    wait(bar(B_SREADY0 + half), t);
                    __syncwarp();
                    tc_fence_after_sync();
#pragma unroll
                    for (int s = 4 * half; s < 4 * half + 4; ++s) s_product(tmem + DS_P, kb, s);
                }
                tc_commit_warp(bar(B_P));
                // O: S x Q, first half
                if (t > 0) wait(bar(B_YFREE), t - 1);
                __syncwarp();
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < DK / 32; ++s) s_product(y, qb, s);
                // (the last M has read its u: U goes over it)
                if (t > 0) wait(bar(B_M0 + ((t - 1) & 1)), (t - 1) >> 1);
                // U: r x T; step s (rows 16 s .. of r) reaches the rows from 16 s on only
                wait(bar(B_RREADY), t);
                __syncwarp();
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t off = static_cast<uint32_t>(2048 * s + 32 * s);
                    const uint64_t hi = desc_mn_sw128(mb + off), lo = desc_mn_sw128(mb + DC_MAT + off);
                    const uint32_t id = tc_idesc_bf16(64 - 16 * s, true), d = tmem + DS_U + 16 * s, r = tmem + DS_R + 8 * s;
                    tc_mma_f16_ts_warp(d, r, hi, id, s > 0);
                    tc_mma_f16_ts_warp(d, r + 32, hi, id, 1);
                    tc_mma_f16_ts_warp(d, r, lo, id, 1);
                }
                tc_commit_warp(bar(B_U));
                // O, second half
#pragma unroll
                for (int s = DK / 32; s < DK / 16; ++s) s_product(y, qb, s);
                // D: u' x K
                wait(bar(B_UREADY), t);
                __syncwarp();
                tc_fence_after_sync();
#pragma unroll
                for (int half = 0; half < HALVES; ++half) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint64_t k = desc_mn_sw128(kb + half * DC_ROWS * 128 + s * 2048);
                        const uint32_t d = tmem + DS_P + 64 * half;
                        tc_mma_f16_ts_warp(d, tmem + DS_UP + 8 * s, k, tc_idesc_bf16(64, true), s > 0);
                        tc_mma_f16_ts_warp(d, tmem + DS_UP + 32 + 8 * s, k, tc_idesc_bf16(64, true), 1);
                    }
                    tc_commit_warp(bar(B_D0 + half));
                }
                // M: u x M
                wait(bar(B_MREADY), t);
                __syncwarp();
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t off = static_cast<uint32_t>(2048 * s + 32 * s);
                    const uint64_t hi = desc_k_sw128(mb + 2 * DC_MAT + off), lo = desc_k_sw128(mb + 3 * DC_MAT + off);
                    const uint32_t id = tc_idesc_bf16(64 - 16 * s, false), d = tmem + DS_M + 16 * s, u = tmem + DS_U + 8 * s;
                    tc_mma_f16_ts_warp(d, u, hi, id, s > 0);
                    tc_mma_f16_ts_warp(d, u + 32, hi, id, 1);
                    tc_mma_f16_ts_warp(d, u, lo, id, 1);
                }
                tc_commit_warp(bar(B_M0 + (t & 1)));
            }
    } else {
        // ------------------------------------------------ conversions
        const int q = warp & 3, h = warp >> 2, l = 32 * q + lane;
        const bool live = l < p.dv;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
        constexpr int SC = DK / 4;              // state columns of a thread
        const int half = h * SC / 64;           // of the state's columns
        constexpr int NTHR = DS_WARPS * 32;
        f32x2 s[SC / 2];
        auto arrive = [&](int i) {              // this warp's tensor memory accesses are done
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };

        // sequences without work: empty ones that start from zero, inactive
        // entries (their outputs are zero)
        for (int b = part; b < cp.B; b += gridDim.x) {
            int bg, en, sl;
            const int nb = w.blocks_of(b, bg, en, sl);
            if (sl >= p.n_slots && threadIdx.x == 0) atomicOr(p.err, 8);
            if (sl < 0 || sl >= p.n_slots) {
                const int per = p.Hv * p.dv / 8;
                for (long long i = threadIdx.x; i < static_cast<long long>(en - bg) * per; i += NTHR)
                    *reinterpret_cast<uint4 *>(p.o + (bg + i / per) * p.ldo + (i % per) * 8) = make_uint4(0u, 0u, 0u, 0u);
            } else if (nb == 0 && cp.zero_init) {
                const long long per = static_cast<long long>(p.Hv) * p.dv * DK;
                for (long long i = threadIdx.x; i < per; i += NTHR) p.state[sl * per + i] = 0.f;
            }
        }

        // Outputs of a step, this thread's rows 16 h .. + 15 of value l: added
        // up as soon as O and M are there, stored later (n rows from o).
        uint32_t outs[8];
        auto take_out = [&](uint32_t t) {
            const float *f = reinterpret_cast<const float *>(ds_smem + L::F + (t & 3) * DC_FACTORS) + 2 * DC_ROWS + 16 * h;
            wait(bar(B_M0 + (t & 1)), t >> 1);      // (and O, issued before it)
            tc_fence_after_sync();
            uint32_t so[16], mo[16];
            tmem_ld<16>(lanes + DS_O + 16 * h, so);
            tmem_ld<16>(lanes + DS_M + 16 * h, mo);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 e = *reinterpret_cast<const float4 *>(f + i);
                outs[i / 2] = pack_bf16x2(fmaf(__uint_as_float(so[i]), e.x, __uint_as_float(mo[i])),
                                          fmaf(__uint_as_float(so[i + 1]), e.y, __uint_as_float(mo[i + 1])));
                outs[i / 2 + 1] = pack_bf16x2(fmaf(__uint_as_float(so[i + 2]), e.z, __uint_as_float(mo[i + 2])),
                                              fmaf(__uint_as_float(so[i + 3]), e.w, __uint_as_float(mo[i + 3])));
            }
            arrive(B_YFREE);
        };
        auto store_out = [&](uint16_t *o, int n) {
            o += 16 * h * p.ldo + l;
            n = live ? n - 16 * h : 0;
            if (n >= 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i, o += p.ldo) *o = static_cast<uint16_t>((i & 1) ? outs[i / 2] >> 16 : outs[i / 2]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i, o += p.ldo)
                    if (i < n) *o = static_cast<uint16_t>((i & 1) ? outs[i / 2] >> 16 : outs[i / 2]);
            }
        };

        uint32_t t = 0, vals[8];
        while (w.next()) {
            float *srow = p.state + ((static_cast<size_t>(w.slot) * p.Hv + w.hv) * p.dv + (live ? l : 0)) * DK + h * SC;
            if (w.takes) {                      // the CTA of the next part hands the state over
                const uint64_t t0 = global_timer_ns();
                while (ld_acquire_gpu_u32(cp.flags + part + 1) == 0u)
                    if (global_timer_ns() - t0 > (*flag ? WAIT_LIMIT_AFTER_ERR_NS : WAIT_LIMIT_NS)) {
                        *flag = 1;
                        atomicOr(p.err, 2);
                        break;
                    }
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < SC; i += 4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live && (w.takes || !cp.zero_init)) v = __ldcg(reinterpret_cast<const float4 *>(srow + i));
                s[i / 2] = pack_x2(v.x, v.y);
                s[i / 2 + 1] = pack_x2(v.z, v.w);
            }
            uint16_t *o = p.o + (static_cast<long long>(w.begin) + static_cast<long long>(w.c0) * DC_ROWS) * p.ldo +
                          static_cast<long long>(w.hv) * p.dv;
            for (int c = w.c0; c < w.c1; ++c, ++t) {
                uint8_t *stage = ds_smem + (t & 1) * L::STAGE;
                const int n = min(DC_ROWS, w.end - w.begin - c * DC_ROWS);
                if (n < DC_ROWS) {
                    // keys past the end are another sequence's and may be NaN: zero
                    wait(bar(B_FULL0 + (t & 1)), t >> 1);
                    for (int i = threadIdx.x; i < (DC_ROWS - n) * (DK / 8); i += NTHR) {
                        const int r = n + i / (DK / 8), j = i % (DK / 8);   // swizzled pieces stay within their row
                        *reinterpret_cast<uint4 *>(stage + L::K + (j >> 3) * DC_ROWS * 128 + r * 128 + (j & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async();
                }
                {   // the state's two terms
                    uint32_t hi[SC / 2], lo[SC / 2];
#pragma unroll
                    for (int i = 0; i < SC / 2; ++i) split_bf16x2(s[i], hi[i], lo[i]);
                    // (the last state's terms have been read: O is issued before D, which has been waited for)
                    tmem_st<SC / 2>(lanes + DS_SHI + h * (SC / 2), hi);
                    tmem_st<SC / 2>(lanes + DS_SLO + h * (SC / 2), lo);
                    arrive(B_SREADY0 + half);
                }
                if (c > w.c0) take_out(t - 1);
                const float *f = reinterpret_cast<const float *>(ds_smem + L::F + (t & 3) * DC_FACTORS);
                uint32_t v[16], hi[8], lo[8];
                // this thread's values, rows in pairs
                auto load_v = [&](uint32_t step) {
                    const uint16_t *vt = reinterpret_cast<const uint16_t *>(ds_smem + (step & 1) * L::STAGE + L::V) + 16 * h * p.dv + (live ? l : 0);
                    wait(bar(B_FULL0 + (step & 1)), step >> 1);
#pragma unroll
                    for (int i = 0; i < 8; ++i) vals[i] = vt[2 * i * p.dv] | (static_cast<uint32_t>(vt[(2 * i + 1) * p.dv]) << 16);
                };
                load_v(t);
                {   // r = v - e^G r_k (S k)
                    wait(bar(B_P), t);
                    tc_fence_after_sync();
                    tmem_ld<16>(lanes + DS_P + 16 * h, v);
                    tmem_wait_ld();
                    f32x2 val[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {        // (the factors are stored negated)
                        const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(f + 16 * h + 2 * i);
                        val[i] = fma_x2(e.x, pair_x2(v[2 * i], v[2 * i + 1]), pair_x2(vals[i] << 16, vals[i] & 0xFFFF0000u));
                        val[i + 1] = fma_x2(e.y, pair_x2(v[2 * i + 2], v[2 * i + 3]), pair_x2(vals[i + 1] << 16, vals[i + 1] & 0xFFFF0000u));
                    }
                    const int m = live ? n - 16 * h : 0;
                    if (m < 16)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (2 * i >= m) val[i] = 0ull;
                            if (2 * i + 1 == m) val[i] &= 0xFFFFFFFFull;
                        }
#pragma unroll
                    for (int i = 0; i < 8; ++i) split_bf16x2(val[i], hi[i], lo[i]);
                    tmem_st<8>(lanes + DS_R + 8 * h, hi);
                    tmem_st<8>(lanes + DS_R + 32 + 8 * h, lo);
                    arrive(B_RREADY);
                }
                if (c > w.c0) {                 // while U runs
                    store_out(o, DC_ROWS);
                    o += DC_ROWS * p.ldo;
                }
                {   // u' = u e^(G_n - G) r_k, and u
                    wait(bar(B_U), t);
                    tc_fence_after_sync();
                    tmem_ld<16>(lanes + DS_U + 16 * h, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(f + DC_ROWS + 16 * h + 2 * i);
                        split_bf16x2(mul_x2(e.x, pair_x2(v[2 * i], v[2 * i + 1])), hi[i], lo[i]);
                        split_bf16x2(mul_x2(e.y, pair_x2(v[2 * i + 2], v[2 * i + 3])), hi[i + 1], lo[i + 1]);
                    }
                    tmem_st<8>(lanes + DS_UP + 8 * h, hi);
                    tmem_st<8>(lanes + DS_UP + 32 + 8 * h, lo);
                    arrive(B_UREADY);
                    // off the chain, while D runs: u's terms over U, which the four
                    // warps of these lanes have read
#pragma unroll
                    for (int i = 0; i < 8; ++i) split_bf16x2(pair_x2(v[2 * i], v[2 * i + 1]), hi[i], lo[i]);
                    tc_fence_before_sync();
                    named_bar_sync(2 + q, 128);
                    tc_fence_after_sync();
                    tmem_st<8>(lanes + DS_U + 8 * h, hi);
                    tmem_st<8>(lanes + DS_U + 32 + 8 * h, lo);
                    arrive(B_MREADY);
                }
                {   // S <- e^(G_n) S + D
                    const f32x2 decay = pack_x2(f[3 * DC_ROWS], f[3 * DC_ROWS]);
                    wait(bar(B_D0 + half), t);
                    tc_fence_after_sync();
#pragma unroll
                    for (int j = 0; j < SC; j += 16) {
                        tmem_ld<16>(lanes + DS_P + h * SC + j, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[j / 2 + i] = fma_x2(decay, s[j / 2 + i], pair_x2(v[2 * i], v[2 * i + 1]));
                    }
                }
            }
            if (live)
#pragma unroll
                for (int i = 0; i < SC; i += 4)
                    *reinterpret_cast<ulonglong2 *>(srow + i) = make_ulonglong2(s[i / 2], s[i / 2 + 1]);
            take_out(t - 1);
            store_out(o, min(DC_ROWS, w.end - w.begin - (w.c1 - 1) * DC_ROWS));
            if (w.gives) {                      // the rest of the chain is the CTA's of the part before
                named_bar_sync(1, NTHR);
                if (threadIdx.x == 0) red_add_release_gpu(cp.flags + part, 1u);
            }
        }
    }
    // every load has landed and every product is done: the warps above have
    // waited for each
    tc_fence_before_sync();
    __syncthreads();
    if (warp == DS_MMA) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, DS_COLS);
    }
}

}  // namespace sv
