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
// two such factors the lo x lo part is left out), so that the state keeps
// fp32-grade accuracy and outputs carry hardly more than their own rounding.
#pragma once

#include <cuda.h>

#include "gated_delta.cuh"
#include "tc_ops.cuh"
#include "w4a16_stream.cuh"

namespace sv {

constexpr int DC_ROWS = 64;                     // rows of a block
constexpr int DC_MAT = DC_ROWS * 128;           // bytes of one 64 x 64 bf16 matrix, 128-byte swizzled
constexpr int DC_FACTORS = 1024;                // bytes of a block's row factors
constexpr int DC_BLOCK = 4 * DC_MAT + DC_FACTORS;   // T (two terms), M (two terms), factors
constexpr float DC_MIN_LOG = -200.f;            // e^-200 is 0 in fp32: a log decay of -inf is taken as this

struct DeltaChunkParams {
    DeltaParams d;                              // rows, shape, state; T and prev unused
    const int32_t *cu;                          // [B + 1] first rows
    int R, B;                                   // rows in all, sequences
    int zero_init;
    uint8_t *ws;                                // [R / 64 + B][Hv][DC_BLOCK]
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

// Row by row, for short sequences.  Grid: x = dv / cols, y = Hv, z = B.
template <int DK>
__global__ void __launch_bounds__(512) gated_delta_rows_kernel(const DeltaChunkParams cp)
{
    extern __shared__ __align__(16) float gd_smem[];
    const DeltaParams &p = cp.d;
    const int cols = p.cols, col0 = blockIdx.x * cols, hv = blockIdx.y, b = blockIdx.z;
    const int i = threadIdx.x & 3, col = threadIdx.x >> 2;
    const GdSmem<DK> sm(gd_smem, GD_MAX_ROWS, cols);
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
        const bool running = gd_stage<DK>(p, p.rows, r0, n, hv, col0, cols, sm, true);
        gd_rows<DK, true>(st, sm, n, cols, running, o, p.ldo);
        o += n * p.ldo;
        __syncthreads();
    }
    st.store(s, i);
}

// ----------------------------------------------------------------- prep

// Byte of element (row, column) of a 64 x 64 bf16 matrix whose 128-byte rows
// are swizzled in 16-byte pieces, as the tensor cores' descriptors expect.
__device__ __forceinline__ int dc_swizzled(int row, int col)
{
    return row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}

template <int DK>
struct DcPrepSmem {
    uint16_t k[DC_ROWS][DK + 8], q[DC_ROWS][DK + 8];
    float a[DC_ROWS][DC_ROWS + 4];
    float rk[DC_ROWS], rq[DC_ROWS], beta[DC_ROWS], g_hi[DC_ROWS], g_lo[DC_ROWS];
    int seq, first, rows;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// Grid: x = R / 64 + B blocks, y = Hv; 128 threads.
template <int DK>
__global__ void __launch_bounds__(128) delta_prep_kernel(const DeltaChunkParams cp)
{
    extern __shared__ __align__(16) uint8_t dc_smem[];
    DcPrepSmem<DK> &sm = *reinterpret_cast<DcPrepSmem<DK> *>(dc_smem);
    const DeltaParams &p = cp.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int id = blockIdx.x, hv = blockIdx.y, hk = hv / (p.Hv / p.Hk);
    pdl_launch_dependents();
    pdl_wait_prior();
    // the sequence whose blocks hold this one (its last row decides where
    // rows are claimed twice, which cu_seqlens must not do)
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
    for (int i = tid; i < DC_ROWS * PR; i += 128) {
        const int t = i / PR, j = (i % PR) * 8;
        uint4 kv = make_uint4(0u, 0u, 0u, 0u), qv = kv;
        if (t < n) {
            kv = __ldg(reinterpret_cast<const uint4 *>(p.rows.k + (row0 + t) * p.rows.ldk + hk * DK + j));
            qv = __ldg(reinterpret_cast<const uint4 *>(p.rows.q + (row0 + t) * p.rows.ldq + hk * DK + j));
        }
        *reinterpret_cast<uint4 *>(&sm.k[t][j]) = kv;
        *reinterpret_cast<uint4 *>(&sm.q[t][j]) = qv;
    }
    // the running sum of the log decays, kept to more than fp32 (differences
    // of large sums give the decays between near rows); two rows a lane
    if (warp == 0) {
        double g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            float v = t < n ? p.rows.g[(row0 + t) * p.rows.ldg + hv] : 0.f;
            if (v < DC_MIN_LOG) v = DC_MIN_LOG;
            g[e] = static_cast<double>(v);
            sm.beta[t] = t < n ? p.rows.beta[(row0 + t) * p.rows.ldg + hv] : 0.f;
        }
        double sum = g[0] + g[1];
        const double own = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double below = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += below;
        }
        const double before = sum - own;
        const double G[2] = {before + g[0], sum};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float hi = static_cast<float>(G[e]);
            sm.g_hi[2 * lane + e] = hi;
            sm.g_lo[2 * lane + e] = static_cast<float>(G[e] - static_cast<double>(hi));
        }
    }
    __syncthreads();
    {   // inverse norms: two threads a row
        const int t = tid >> 1, c0 = (tid & 1) * (DK / 2);
        float kk = 0.f, qq = 0.f;
#pragma unroll 8
        for (int c = 0; c < DK / 2; ++c) {
            const float kf = bf16_bits_to_float(sm.k[t][c0 + c]), qf = bf16_bits_to_float(sm.q[t][c0 + c]);
            kk = fmaf(kf, kf, kk);
            qq = fmaf(qf, qf, qq);
        }
        kk += __shfl_xor_sync(0xFFFFFFFFu, kk, 1);
        qq += __shfl_xor_sync(0xFFFFFFFFu, qq, 1);
        if ((tid & 1) == 0) {
            sm.rk[t] = p.l2norm ? 1.f / sqrtf(kk + GD_L2_EPS) : 1.f;
            sm.rq[t] = p.scale * (p.l2norm ? 1.f / sqrtf(qq + GD_L2_EPS) : 1.f);
        }
    }
    __syncthreads();
    // k_i . k_j and q_i . k_j: a warp has 16 rows i of both
    float ck[8][4], cq[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) ck[j][e] = cq[j][e] = 0.f;
    const uint32_t arow = static_cast<uint32_t>(((warp * 16 + (lane & 15)) * (DK + 8) + (lane >> 4) * 8) * 2);
    const uint32_t brow = static_cast<uint32_t>((((lane & 7) + ((lane >> 4) << 3)) * (DK + 8) + ((lane >> 3) & 1) * 8) * 2);
    const uint32_t k0 = smem_addr(&sm.k[0][0]), q0 = smem_addr(&sm.q[0][0]);
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        uint32_t ak[4], aq[4];
        ldmatrix_x4(ak, k0 + arow + 32u * s);
        ldmatrix_x4(aq, q0 + arow + 32u * s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t b[4];
            ldmatrix_x4(b, k0 + brow + static_cast<uint32_t>(j * 16 * (DK + 8) * 2) + 32u * s);
            mma_bf16_16816(ck[2 * j], ak[0], ak[1], ak[2], ak[3], b[0], b[1]);
            mma_bf16_16816(ck[2 * j + 1], ak[0], ak[1], ak[2], ak[3], b[2], b[3]);
            mma_bf16_16816(cq[2 * j], aq[0], aq[1], aq[2], aq[3], b[0], b[1]);
            mma_bf16_16816(cq[2 * j + 1], aq[0], aq[1], aq[2], aq[3], b[2], b[3]);
        }
    }
    uint8_t *out = cp.ws + (static_cast<size_t>(id) * p.Hv + hv) * DC_BLOCK;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = warp * 16 + (lane >> 2) + 8 * h;
        const float gi = sm.g_hi[i], gl = sm.g_lo[i], bi = sm.beta[i] * sm.rk[i], qi = sm.rq[i];
#pragma unroll
        for (int j8 = 0; j8 < 8; ++j8) {
            float m[2];
            const int j0 = j8 * 8 + (lane & 3) * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = j0 + e;
                float d = 0.f;
                if (j <= i && i < n) d = expf((gi - sm.g_hi[j]) + (gl - sm.g_lo[j])) * sm.rk[j];
                m[e] = j <= i && i < n ? cq[j8][2 * h + e] * d * qi : 0.f;
                sm.a[i][j] = j < i && i < n ? ck[j8][2 * h + e] * d * bi : 0.f;
            }
            uint32_t hi, lo;
            split_bf16x2(m[0], m[1], hi, lo);
            *reinterpret_cast<uint32_t *>(out + 2 * DC_MAT + dc_swizzled(i, j0)) = hi;
            *reinterpret_cast<uint32_t *>(out + 3 * DC_MAT + dc_swizzled(i, j0)) = lo;
        }
    }
    if (tid < DC_ROWS) {
        // row factors: e^G r_k, e^(G_n - G) r_k, scale e^G r_q; the block's decay
        float *f = reinterpret_cast<float *>(out + 4 * DC_MAT);
        const float g = sm.g_hi[tid], gl = sm.g_lo[tid], e = expf(g + gl);
        const float last = expf((sm.g_hi[DC_ROWS - 1] - g) + (sm.g_lo[DC_ROWS - 1] - gl));
        f[tid] = tid < n ? e * sm.rk[tid] : 0.f;
        f[DC_ROWS + tid] = tid < n ? last * sm.rk[tid] : 0.f;
        f[2 * DC_ROWS + tid] = tid < n ? e * sm.rq[tid] : 0.f;
        if (tid == 0) f[3 * DC_ROWS] = expf(sm.g_hi[DC_ROWS - 1] + sm.g_lo[DC_ROWS - 1]);
    }
    __syncthreads();
    if (tid < DC_ROWS) {
        // column tid of (I + A)^-1 by forward substitution, in registers
        float t[DC_ROWS];
#pragma unroll
        for (int i = 0; i < DC_ROWS; ++i) {
            float s0 = i == tid ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int m = 0; m + 3 < i; m += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&sm.a[i][m]);
                s0 = fmaf(-a.x, t[m], s0);
                s1 = fmaf(-a.y, t[m + 1], s1);
                s2 = fmaf(-a.z, t[m + 2], s2);
                s3 = fmaf(-a.w, t[m + 3], s3);
            }
#pragma unroll
            for (int m = i & ~3; m < i; ++m) s0 = fmaf(-sm.a[i][m], t[m], s0);
            t[i] = (s0 + s1) + (s2 + s3);
        }
        const float b = sm.beta[tid];
#pragma unroll
        for (int i = 0; i < DC_ROWS; ++i) {
            uint32_t hi, lo;
            split_bf16x2(t[i] * b, 0.f, hi, lo);
            *reinterpret_cast<uint16_t *>(out + dc_swizzled(i, tid)) = static_cast<uint16_t>(hi);
            *reinterpret_cast<uint16_t *>(out + DC_MAT + dc_swizzled(i, tid)) = static_cast<uint16_t>(lo);
        }
    }
}

// ----------------------------------------------------------------- scan
//
// One CTA per head and sequence.  Everything is transposed, with the value
// dimension on the tensor memory's lanes (state row l on lane l), so that the
// state, r and u are A operands in tensor memory and the keys, queries, T and
// M are B operands in shared memory exactly as they are loaded.
//
//   phase  product                               accumulator
//   P      S (2 terms) x K                       X
//   O      S (2) x Q                             Y
//   U      r (2) x T (2), without lo x lo        S_hi
//   M      u (2) x M (2), without lo x lo        Y, after scaling its columns
//   D      u' (2) x K, 64 keys' columns each     S_hi and X
//
// Warps 0-7 convert: warp w has lanes 32 (w & 3) .. + 31, half w >> 2 of the
// columns; the state's fp32 values stay in their registers.  Warp 8 issues
// the loads and the products.  Tensor memory: S_hi, S_lo (64 columns each,
// the state's two terms; later u's accumulator and u''s two terms), X (64: P,
// then r's two terms, then u's, then the second half of D) and Y (64): 256
// columns and 98 KB of shared memory, so that two CTAs share an SM and one
// computes while the other converts.

constexpr int DS_THREADS = 288;
constexpr uint32_t DS_COLS = 256;
constexpr uint32_t DS_SHI = 0, DS_SLO = 64, DS_X = 128, DS_Y = 192;

template <int DK>
struct DsSmem {                                 // from a 1024-byte boundary
    static constexpr int TILE = DC_ROWS * DK * 2;   // keys or queries: DK / 64 boxes of [64 rows][128 bytes]
    static constexpr int K = 0;                 // two buffers
    static constexpr int Q = K + 2 * TILE;
    static constexpr int MATS = Q + TILE;       // T hi, T lo, M hi, M lo
    static constexpr int V = MATS + 4 * DC_MAT; // [64][dv]
    static constexpr int F = V + DC_ROWS * 128 * 2;     // two buffers of row factors
    static constexpr int BARS = F + 2 * DC_FACTORS;
    static constexpr int BYTES = BARS + 256;
};

enum { B_K0, B_K1, B_F0, B_F1, B_V, B_Q, B_T, B_M, B_SREADY, B_RREADY, B_UREADY, B_YFREE, B_P, B_O, B_U, B_MO, B_D, B_COUNT };

constexpr uint32_t ds_idesc(int n, bool b_mn)
{
    // fp32 accumulator, bf16 operands; B along the rows' length (K-major) or across
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           ((128u >> 4) << 24);
}

struct DsWait {
    volatile int *flag;
    int *err;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const
    {
        if (mbar_try_wait(bar, parity & 1u)) return;
        if (!mbar_wait_bounded(bar, parity & 1u, *flag ? WAIT_LIMIT_AFTER_ERR_NS : WAIT_LIMIT_NS)) {
            *flag = 1;
            atomicOr(err, 2);
        }
    }
};

template <int DK>
__global__ void __launch_bounds__(DS_THREADS, 2)
delta_scan_kernel(const __grid_constant__ DeltaChunkParams cp, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmV)
{
    extern __shared__ __align__(1024) uint8_t ds_smem[];
    using L = DsSmem<DK>;
    const DeltaParams &p = cp.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hv = blockIdx.x, b = blockIdx.y, hk = hv / (p.Hv / p.Hk);
    const uint32_t base = smem_addr(ds_smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ds_smem + L::BARS);
    volatile int *flag = reinterpret_cast<volatile int *>(bars + B_COUNT);
    volatile uint32_t *slot_tm = reinterpret_cast<volatile uint32_t *>(flag + 1);
    auto bar = [&](int i) { return base + static_cast<uint32_t>(L::BARS + 8 * i); };
    const DsWait wait{flag, p.err};

    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.err, 4);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), i >= B_SREADY && i <= B_YFREE ? 8 : 1);
        *flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_addr(const_cast<uint32_t *>(slot_tm)), DS_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *slot_tm;
    pdl_launch_dependents();
    pdl_wait_prior();

    int begin, end;
    gd_range(cp.cu, cp.R, b, begin, end);
    const int slot = gd_slot(p.state_idx, p.n_slots, b, p.err);
    const int chunks = slot < 0 ? 0 : (end - begin + DC_ROWS - 1) / DC_ROWS;
    const uint8_t *blocks = cp.ws + (static_cast<size_t>(dc_base(begin, b)) * p.Hv + hv) * DC_BLOCK;
    const size_t block_step = static_cast<size_t>(p.Hv) * DC_BLOCK;

    if (warp == 8) {
        // ------------------------------------------------ loads and products
        const uint64_t keep = policy_evict_last(), once = policy_evict_first();
        auto load_rows = [&](const CUtensorMap &m, int dst, int bar_i, int c, int col, int width, bool swizzled) {
            // 64 rows from block c; rows past the end are another sequence's
            mbar_arrive_expect_tx(bar(bar_i), static_cast<uint32_t>(DC_ROWS * width * 2));
            if (swizzled) {
#pragma unroll
                for (int j = 0; j < DK / 64; ++j)
                    tma_load_2d(base + dst + j * DC_ROWS * 128, &m, col + 64 * j, begin + c * DC_ROWS, bar(bar_i), keep);
            } else {
                tma_load_2d(base + dst, &m, col, begin + c * DC_ROWS, bar(bar_i), once);
            }
        };
        auto load_k = [&](int c) { load_rows(tmK, L::K + (c & 1) * L::TILE, B_K0 + (c & 1), c, hk * DK, DK, true); };
        auto load_f = [&](int c) {
            mbar_arrive_expect_tx(bar(B_F0 + (c & 1)), DC_FACTORS);
            bulk_g2s(base + L::F + (c & 1) * DC_FACTORS, blocks + c * block_step + 4 * DC_MAT, DC_FACTORS,
                     bar(B_F0 + (c & 1)), once);
        };
        auto load_v = [&](int c) { load_rows(tmV, L::V, B_V, c, hv * p.dv, p.dv, false); };
        auto load_q = [&](int c) { load_rows(tmQ, L::Q, B_Q, c, hk * DK, DK, true); };
        auto load_mats = [&](int c, int which) {    // 0: T, 1: M
            mbar_arrive_expect_tx(bar(B_T + which), 2 * DC_MAT);
            bulk_g2s(base + L::MATS + which * 2 * DC_MAT, blocks + c * block_step + which * 2 * DC_MAT, 2 * DC_MAT,
                     bar(B_T + which), once);
        };
        if (lane == 0 && chunks > 0) {
            load_k(0);
            load_f(0);
            load_v(0);
            load_q(0);
            load_mats(0, 0);
            load_mats(0, 1);
            if (chunks > 1) {
                load_k(1);
                load_f(1);
            }
        }
        __syncwarp();
        const uint32_t shi = tmem + DS_SHI, slo = tmem + DS_SLO, x = tmem + DS_X, y = tmem + DS_Y;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = static_cast<uint32_t>(c);
            const uint32_t kb = base + static_cast<uint32_t>(L::K + (c & 1) * L::TILE), qb = base + L::Q;
            const bool more = c + 1 < chunks;
            // P: S x K
            wait(bar(B_SREADY), ph);
            if (lane == 0 && c > 0 && more) {       // block c - 1 is done with its keys and factors
                load_k(c + 1);
                load_f(c + 1);
            }
            wait(bar(B_K0 + (c & 1)), ph >> 1);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                const uint64_t d = desc_k_sw128(kb + (s >> 2) * DC_ROWS * 128 + (s & 3) * 32);
                tc_mma_f16_ts_warp(x, shi + 8 * s, d, ds_idesc(64, false), s > 0);
                tc_mma_f16_ts_warp(x, slo + 8 * s, d, ds_idesc(64, false), 1);
            }
            tc_commit_warp(bar(B_P));
            // O: S x Q
            if (c > 0) wait(bar(B_YFREE), ph - 1);
            wait(bar(B_Q), ph);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                const uint64_t d = desc_k_sw128(qb + (s >> 2) * DC_ROWS * 128 + (s & 3) * 32);
                tc_mma_f16_ts_warp(y, shi + 8 * s, d, ds_idesc(64, false), s > 0);
                tc_mma_f16_ts_warp(y, slo + 8 * s, d, ds_idesc(64, false), 1);
            }
            tc_commit_warp(bar(B_O));
            // U: r x T; T is lower triangular, so step s (rows 16 s .. of r)
            // reaches the rows from 16 s on only
            wait(bar(B_RREADY), ph);
            if (lane == 0 && more) load_v(c + 1);
            wait(bar(B_O), ph);                     // S_hi is free
            if (lane == 0 && more) load_q(c + 1);
            wait(bar(B_T), ph);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t off = static_cast<uint32_t>(16 * s * 128 + 32 * s);
                const uint64_t hi = desc_k_sw128(base + L::MATS + off), lo = desc_k_sw128(base + L::MATS + DC_MAT + off);
                const uint32_t id = ds_idesc(64 - 16 * s, false), d = shi + 16 * s;
                tc_mma_f16_ts_warp(d, x + 8 * s, hi, id, s > 0);
                tc_mma_f16_ts_warp(d, x + 32 + 8 * s, hi, id, 1);
                tc_mma_f16_ts_warp(d, x + 8 * s, lo, id, 1);
            }
            tc_commit_warp(bar(B_U));
            // M: u x M on top of the scaled S x Q
            wait(bar(B_UREADY), ph);
            if (lane == 0 && more) load_mats(c + 1, 0);
            wait(bar(B_M), ph);
            __syncwarp();
            tc_fence_after_sync();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t off = static_cast<uint32_t>(16 * s * 128 + 32 * s);
                const uint32_t id = ds_idesc(64 - 16 * s, false), d = y + 16 * s;
                const uint64_t hi = desc_k_sw128(base + L::MATS + 2 * DC_MAT + off), lo = desc_k_sw128(base + L::MATS + 3 * DC_MAT + off);
                tc_mma_f16_ts_warp(d, x + 8 * s, hi, id, 1);
                tc_mma_f16_ts_warp(d, x + 32 + 8 * s, hi, id, 1);
                tc_mma_f16_ts_warp(d, x + 8 * s, lo, id, 1);
            }
            tc_commit_warp(bar(B_MO));
            // D: u' x K, the key columns 0..63, then 64..127 over u
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint64_t d = desc_mn_sw128(kb + s * 2048);
                tc_mma_f16_ts_warp(shi, slo + 8 * s, d, ds_idesc(64, true), s > 0);
                tc_mma_f16_ts_warp(shi, slo + 32 + 8 * s, d, ds_idesc(64, true), 1);
            }
            wait(bar(B_MO), ph);
            if (lane == 0 && more) load_mats(c + 1, 1);
            __syncwarp();
            if (DK == 128) {
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint64_t d = desc_mn_sw128(kb + DC_ROWS * 128 + s * 2048);
                    tc_mma_f16_ts_warp(x, slo + 8 * s, d, ds_idesc(64, true), s > 0);
                    tc_mma_f16_ts_warp(x, slo + 32 + 8 * s, d, ds_idesc(64, true), 1);
                }
            }
            tc_commit_warp(bar(B_D));
        }
    } else {
        // ------------------------------------------------ conversions
        const int q = warp & 3, h = warp >> 2, l = 32 * q + lane;
        const bool live = l < p.dv;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
        constexpr int SC = DK / 2;              // state columns of a thread
        float st[SC];
        const size_t srow = ((static_cast<size_t>(slot < 0 ? 0 : slot) * p.Hv + hv) * p.dv + (live ? l : 0)) * DK + h * SC;
#pragma unroll
        for (int i = 0; i < SC; i += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live && slot >= 0 && !cp.zero_init) v = *reinterpret_cast<const float4 *>(p.state + srow + i);
            st[i] = v.x;
            st[i + 1] = v.y;
            st[i + 2] = v.z;
            st[i + 3] = v.w;
        }
        uint16_t *o = p.o + static_cast<long long>(begin) * p.ldo + static_cast<long long>(hv) * p.dv;
        auto arrive = [&](int i) {              // this warp's tensor memory accesses are done
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        auto pair_sync = [&]() {                // the two warps of these lanes
            tc_fence_before_sync();
            named_bar_sync(1 + q, 64);
            tc_fence_after_sync();
        };
        // outputs of block c: this thread's rows 32 h .. + 31 of value l;
        // two lanes trade so that each stores pairs of values
        auto store_out = [&](int c) {
            wait(bar(B_MO), static_cast<uint32_t>(c));
            tc_fence_after_sync();
            uint32_t v[32];
            tmem_ld32(lanes + DS_Y + 32 * h, v);
            tmem_wait_ld();
            arrive(B_YFREE);
            const int n = min(DC_ROWS, end - begin - c * DC_ROWS);
            uint16_t *oc = o + static_cast<long long>(c) * DC_ROWS * p.ldo + (l & ~1);
            const bool odd = lane & 1;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float give = __uint_as_float(odd ? v[i] : v[i + 1]), own = __uint_as_float(odd ? v[i + 1] : v[i]);
                const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
                const int t = 32 * h + i + (odd ? 1 : 0);
                if (live && t < n) *reinterpret_cast<uint32_t *>(oc + t * p.ldo) = odd ? pack_bf16x2(got, own) : pack_bf16x2(own, got);
            }
        };
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = static_cast<uint32_t>(c);
            const int n = min(DC_ROWS, end - begin - c * DC_ROWS);
            if (n < DC_ROWS) {
                // keys past the end are another sequence's and may be NaN: zero
                wait(bar(B_K0 + (c & 1)), ph >> 1);
                uint8_t *kt = ds_smem + L::K + (c & 1) * L::TILE;
                for (int i = threadIdx.x; i < (DC_ROWS - n) * (DK / 8); i += 256) {
                    const int t = n + i / (DK / 8), j = i % (DK / 8);   // swizzled pieces stay within their row
                    *reinterpret_cast<uint4 *>(kt + (j >> 3) * DC_ROWS * 128 + t * 128 + (j & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
            }
            {   // the state's two terms
                uint32_t hi[SC / 2], lo[SC / 2];
#pragma unroll
                for (int i = 0; i < SC / 2; ++i) split_bf16x2(st[2 * i], st[2 * i + 1], hi[i], lo[i]);
                tmem_st<SC / 2>(lanes + DS_SHI + h * (SC / 2), hi);
                tmem_st<SC / 2>(lanes + DS_SLO + h * (SC / 2), lo);
                arrive(B_SREADY);
            }
            if (c > 0) store_out(c - 1);
            const float *f = reinterpret_cast<const float *>(ds_smem + L::F + (c & 1) * DC_FACTORS);
            wait(bar(B_F0 + (c & 1)), ph >> 1);
            wait(bar(B_V), ph);
            {   // r = v - e^G r_k (S k)
                const uint16_t *vt = reinterpret_cast<const uint16_t *>(ds_smem + L::V) + 32 * h * p.dv + (live ? l : 0);
                wait(bar(B_P), ph);
                tc_fence_after_sync();
                uint32_t v[32], hi[16], lo[16];
                tmem_ld32(lanes + DS_X + 32 * h, v);
                tmem_wait_ld();
                pair_sync();                    // both have read P: r goes over it
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float r[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 32 * h + i + e;
                        r[e] = live && t < n ? fmaf(-f[t], __uint_as_float(v[i + e]), bf16_bits_to_float(vt[(i + e) * p.dv])) : 0.f;
                    }
                    split_bf16x2(r[0], r[1], hi[i / 2], lo[i / 2]);
                }
                tmem_st<16>(lanes + DS_X + 16 * h, hi);
                tmem_st<16>(lanes + DS_X + 32 + 16 * h, lo);
                arrive(B_RREADY);
            }
            {   // scale the columns of S q while r x T runs
                wait(bar(B_O), ph);
                tc_fence_after_sync();
                uint32_t v[32];
                tmem_ld32(lanes + DS_Y + 32 * h, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f[2 * DC_ROWS + 32 * h + i]);
                tmem_st<32>(lanes + DS_Y + 32 * h, v);
            }
            {   // u, and u' = u e^(G_n - G) r_k in two terms
                wait(bar(B_U), ph);
                tc_fence_after_sync();
                uint32_t v[32], w[16], lo[16];
                tmem_ld32(lanes + DS_SHI + 32 * h, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    split_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), w[i], lo[i]);
                tmem_st<16>(lanes + DS_X + 16 * h, w);
                tmem_st<16>(lanes + DS_X + 32 + 16 * h, lo);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = 32 * h + 2 * i;
                    split_bf16x2(__uint_as_float(v[2 * i]) * f[DC_ROWS + t], __uint_as_float(v[2 * i + 1]) * f[DC_ROWS + t + 1], w[i], lo[i]);
                }
                tmem_st<16>(lanes + DS_SLO + 16 * h, w);
                tmem_st<16>(lanes + DS_SLO + 32 + 16 * h, lo);
                arrive(B_UREADY);
            }
            {   // S <- e^(G_n) S + D
                const float decay = f[3 * DC_ROWS];
                wait(bar(B_D), ph);
                tc_fence_after_sync();
                const uint32_t from = DK == 128 ? (h ? DS_X : DS_SHI) : DS_SHI + 32 * h;
#pragma unroll
                for (int j = 0; j < SC; j += 32) {
                    uint32_t v[32];
                    tmem_ld32(lanes + from + j, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) st[j + i] = fmaf(decay, st[j + i], __uint_as_float(v[i]));
                }
                pair_sync();                    // both have read D: the state's terms go over it
            }
        }
        if (chunks > 0) store_out(chunks - 1);
        if (slot >= 0) {
            if (live && (chunks > 0 || cp.zero_init))
#pragma unroll
                for (int i = 0; i < SC; i += 4)
                    *reinterpret_cast<float4 *>(p.state + srow + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
        } else if (live) {                      // an inactive entry: its outputs are zero
            for (int t = begin + h; t < end; t += 2, o += 2 * p.ldo) o[h * p.ldo + l] = 0;
        }
    }
    // every load has landed (each was waited for) and every product is done
    // (the last commit was waited for by the warps above)
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, DS_COLS);
    }
}

}  // namespace sv
