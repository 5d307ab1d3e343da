// gated_delta.cuh -- the gated delta rule row by row, for decode and verify
// rows.
//
// Each value head keeps a state S of dv rows and dk columns (fp32).  A row
// with key k, query q, value v, log decay g and rate beta does
//
//   S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q
//
// The dv rows of S never mix, so a block takes 32 of them of one head of
// one sequence and a thread a quarter of one: DK / 4 state values in
// registers, read and written once.  Four lanes share a row of S, and each
// takes every fourth 16-byte piece of it, so that a warp's access is eight
// 64-byte runs and the keys in shared memory are read as one broadcast run.
//
// The decay is not applied to every state value of every row: with c the
// product of the decays so far, the registers hold S / c, so a row costs two
// fused multiply-adds a value (S k and the update), three with a query --
// S q is taken before the update and completed with q.k:
//   o = scale (c (S/c) q + u (q.k)),  S/c <- S/c + (u / c) k^T.
// They run two values at a time (fma.rn.f32x2).  A block of rows whose decays
// multiply up to beyond e^+-10 applies each decay at once instead.
//
// A verify cycle's rows are provisional until the head has said how many
// drafts hold.  So the state is not advanced past them: the next cycle's call
// brings the last cycle's rows again (prev) with accept_len, replays the
// accepted ones into the state, writes it, and runs the new rows on from
// there without writing -- one state read and one state write a cycle, and no
// snapshots.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "sv_ptx.cuh"

namespace sv {

constexpr int GD_MAX_ROWS = 32;                 // rows of one staged block
constexpr int GD_COLS = 32, GD_THREADS = 4 * GD_COLS;   // state rows of a block
constexpr int gd_blocks(int dk) { return 512 / dk; }    // of a multiprocessor: DK registers a thread
constexpr float GD_MAX_LOG = 10.f;              // largest |sum of log decays| kept outside the state
constexpr float GD_L2_EPS = 1e-6f;
constexpr float GD_MIN_LOG = -200.f;            // e^-200 is 0 in fp32: a log decay of -inf is taken as this by the block forms

struct DeltaRows {
    const uint16_t *q, *k, *v;                  // bf16 bits, [rows][heads][d]
    const float *g, *beta;                      // [rows][Hv]
    long long ldq, ldk, ldv, ldg;               // elements from row to row
};

struct DeltaParams {
    DeltaRows rows, prev;
    int T, prev_T;                              // rows of a sequence, rows of its last block (0: none)
    const int32_t *accept_len;                  // null: all of prev is replayed
    int Hk, Hv, dv;
    float scale;
    int l2norm, commit;
    float *state;                               // [n_slots][Hv][dv][DK]
    const int32_t *state_idx;                   // null: sequence b has slot b
    int n_slots;
    uint16_t *o;
    long long ldo;
    int *err;
};

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 fma_x2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ f32x2 mul_x2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ f32x2 pack_x2(float lo, float hi)
{
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ float sum_x2(f32x2 a)
{
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
    return lo + hi;
}

__device__ __forceinline__ ulonglong2 lds_x4(uint32_t addr)
{
    ulonglong2 v;
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(addr));
    return v;
}

// Shared memory of a block (floats): keys and queries [GD][DK] each, values
// [GD][GD_COLS], then per row beta, e^g, the running decay, its inverse, q.k.
__host__ __device__ constexpr int gd_smem_floats(int rows, int dk) { return rows * (2 * dk + GD_COLS + 5); }

template <int DK>
struct GdSmem {
    float *k, *q, *v, *beta, *eg, *c, *cinv, *qk;
    __device__ __forceinline__ GdSmem(float *base, int rows)
    {
        k = base;
        q = k + rows * DK;
        v = q + rows * DK;
        beta = v + rows * GD_COLS;
        eg = beta + rows;
        c = eg + rows;
        cinv = c + rows;
        qk = cinv + rows;
    }
};

// What a thread reads first of a block of rows: its values of the warp's first
// row, its first values, the gates of a row (the last warp).
template <int DK>
struct GdFirst {
    uint32_t k[DK / 64], q[DK / 64];
    uint4 v;
    float g, beta;
};

template <int N>
__device__ __forceinline__ void gd_read(const uint16_t *src, uint32_t (&d)[N])
{
    if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(src);
        d[0] = u.x;
        d[1] = u.y;
    } else {
        d[0] = *reinterpret_cast<const uint32_t *>(src);
    }
}

template <int DK>
__device__ __forceinline__ void gd_first(const DeltaParams &p, const DeltaRows &r, long long r0, int n, int hv, int col0,
                                         bool want_q, GdFirst<DK> &f)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hk = hv / (p.Hv / p.Hk);
    if (warp < n) {
        gd_read(r.k + (r0 + warp) * r.ldk + static_cast<long long>(hk) * DK + lane * (DK / 32), f.k);
        if (want_q) gd_read(r.q + (r0 + warp) * r.ldq + static_cast<long long>(hk) * DK + lane * (DK / 32), f.q);
    }
    if (tid < n * (GD_COLS / 8)) {
        const int t = tid / (GD_COLS / 8), j = tid % (GD_COLS / 8) * 8;
        f.v = *reinterpret_cast<const uint4 *>(r.v + (r0 + t) * r.ldv + static_cast<long long>(hv) * p.dv + col0 + j);
    }
    if (warp == GD_THREADS / 32 - 1 && lane < n) {
        f.g = r.g[(r0 + lane) * r.ldg + hv];
        f.beta = r.beta[(r0 + lane) * r.ldg + hv];
    }
}

// Stage `n` rows (first row r0) of head hv in shared memory, `f` of them
// having been read: keys and queries in fp32 (normalised where asked, the
// query times `scale`), q.k, this block's values, the gates and their running
// products.  Returns whether the running products may be used (uniform over
// the block).
template <int DK>
__device__ __forceinline__ bool gd_stage(const DeltaParams &p, const DeltaRows &r, long long r0, int n, int hv, int col0,
                                         const GdSmem<DK> &sm, bool want_q, const GdFirst<DK> &f)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NWARP = GD_THREADS / 32;
    constexpr int E = DK / 32;                  // a lane's values of a row, consecutive
    const int hk = hv / (p.Hv / p.Hk);
    for (int t = warp; t < n; t += NWARP) {
        uint32_t kw[E / 2], qw[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            kw[e] = f.k[e];
            qw[e] = want_q ? f.q[e] : 0u;
        }
        if (t != warp) {
            gd_read(r.k + (r0 + t) * r.ldk + static_cast<long long>(hk) * DK + lane * E, kw);
            if (want_q) gd_read(r.q + (r0 + t) * r.ldq + static_cast<long long>(hk) * DK + lane * E, qw);
        }
        float k[E], q[E];
        float kk = 0.f, qq = 0.f, qk = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            k[e] = __uint_as_float((e & 1) ? kw[e / 2] & 0xFFFF0000u : kw[e / 2] << 16);
            q[e] = __uint_as_float((e & 1) ? qw[e / 2] & 0xFFFF0000u : qw[e / 2] << 16);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            kk = fmaf(k[e], k[e], kk);
            qq = fmaf(q[e], q[e], qq);
            qk = fmaf(q[e], k[e], qk);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            kk += __shfl_xor_sync(0xFFFFFFFFu, kk, o);
            qq += __shfl_xor_sync(0xFFFFFFFFu, qq, o);
            qk += __shfl_xor_sync(0xFFFFFFFFu, qk, o);
        }
        const float rk = p.l2norm ? 1.f / sqrtf(kk + GD_L2_EPS) : 1.f;
        const float rq = p.scale * (p.l2norm ? 1.f / sqrtf(qq + GD_L2_EPS) : 1.f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sm.k[t * DK + lane * E + e] = k[e] * rk;
            if (want_q) sm.q[t * DK + lane * E + e] = q[e] * rq;
        }
        if (lane == 0) sm.qk[t] = qk * rk * rq;
    }
    // values: eight per thread
    for (int i = tid; i < n * (GD_COLS / 8); i += GD_THREADS) {
        const int t = i / (GD_COLS / 8), j = i % (GD_COLS / 8) * 8;
        const uint4 u = i == tid ? f.v : *reinterpret_cast<const uint4 *>(r.v + (r0 + t) * r.ldv + static_cast<long long>(hv) * p.dv + col0 + j);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sm.v[t * GD_COLS + j + 2 * e] = __uint_as_float(w[e] << 16);
            sm.v[t * GD_COLS + j + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    // gates; the running sum of the log decays by a warp scan (n <= 32)
    bool ok = true;
    if (warp == NWARP - 1) {
        const float g = lane < n ? f.g : 0.f;
        float G = g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float below = __shfl_up_sync(0xFFFFFFFFu, G, o);
            if (lane >= o) G += below;
        }
        ok = !(fabsf(G) > GD_MAX_LOG);          // (a NaN spoils its row and later ones either way)
        if (lane < n) {
            sm.beta[lane] = f.beta;
            sm.eg[lane] = expf(g);
            sm.c[lane] = expf(G);
            sm.cinv[lane] = expf(-G);
        }
    }
    return __syncthreads_and(ok) != 0;
}

// One thread's quarter of a state row: piece m (0 .. DK / 16 - 1) holds
// columns 16 m + 4 i .. + 3 as two f32x2, i = lane & 3.
template <int DK>
struct GdState {
    f32x2 s[DK / 8];

    __device__ __forceinline__ void load(const float *p, int i)
    {
#pragma unroll
        for (int m = 0; m < DK / 16; ++m) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p + 16 * m + 4 * i);
            s[2 * m] = v.x;
            s[2 * m + 1] = v.y;
        }
    }
    __device__ __forceinline__ void store(float *p, int i) const
    {
#pragma unroll
        for (int m = 0; m < DK / 16; ++m)
            *reinterpret_cast<ulonglong2 *>(p + 16 * m + 4 * i) = make_ulonglong2(s[2 * m], s[2 * m + 1]);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int m = 0; m < DK / 8; ++m) s[m] = 0ull;
    }
    __device__ __forceinline__ void scale(float c)
    {
        const f32x2 c2 = pack_x2(c, c);
#pragma unroll
        for (int m = 0; m < DK / 8; ++m) s[m] = mul_x2(s[m], c2);
    }
};

// Run `n` staged rows through the state.  OUT: write their outputs (to
// o + t * ldo, bf16).  Afterwards the registers hold S itself.
template <int DK, bool OUT>
__device__ __forceinline__ void gd_rows(GdState<DK> &st, const GdSmem<DK> &sm, int n, bool running,
                                        uint16_t *o, long long ldo)
{
    const int i = threadIdx.x & 3, col = threadIdx.x >> 2;
    const uint32_t ka = smem_addr(sm.k) + 16u * static_cast<uint32_t>(i);
    const uint32_t qa = smem_addr(sm.q) + 16u * static_cast<uint32_t>(i);
    for (int t = 0; t < n; ++t) {
        float c = sm.c[t], cinv = sm.cinv[t];
        if (!running) {
            st.scale(sm.eg[t]);
            c = cinv = 1.f;
        }
        f32x2 k[DK / 8];
        f32x2 a0 = 0ull, a1 = 0ull, b0 = 0ull, b1 = 0ull;
#pragma unroll
        for (int m = 0; m < DK / 16; ++m) {
            const ulonglong2 kv = lds_x4(ka + static_cast<uint32_t>(4 * DK * t + 64 * m));
            k[2 * m] = kv.x;
            k[2 * m + 1] = kv.y;
            a0 = fma_x2(st.s[2 * m], kv.x, a0);
            a1 = fma_x2(st.s[2 * m + 1], kv.y, a1);
            if (OUT) {
                const ulonglong2 qv = lds_x4(qa + static_cast<uint32_t>(4 * DK * t + 64 * m));
                b0 = fma_x2(st.s[2 * m], qv.x, b0);
                b1 = fma_x2(st.s[2 * m + 1], qv.y, b1);
            }
        }
        float a = sum_x2(a0) + sum_x2(a1);
        float b = OUT ? sum_x2(b0) + sum_x2(b1) : 0.f;
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
            if (OUT) b += __shfl_xor_sync(0xFFFFFFFFu, b, d);
        }
        const float u = sm.beta[t] * (sm.v[t * GD_COLS + col] - c * a);
        if (OUT && i == 0) o[t * ldo + col] = __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(c, b, u * sm.qk[t])));
        const float uc = u * cinv;
        const f32x2 u2 = pack_x2(uc, uc);
#pragma unroll
        for (int m = 0; m < DK / 8; ++m) st.s[m] = fma_x2(u2, k[m], st.s[m]);
    }
    if (running && n > 0) st.scale(sm.c[n - 1]);
}

// The slot of sequence b, or -1 when it has none (a negative index) or the
// index is out of range (the error word then says so).
__device__ __forceinline__ int gd_slot(const int32_t *state_idx, int n_slots, int b, int *err)
{
    const int slot = state_idx ? state_idx[b] : b;
    if (slot < n_slots) return slot;
    if (threadIdx.x == 0) atomicOr(err, 8);
    return -1;
}

// One or two rows in all.  Grid: x = dv / GD_COLS, y = Hv, z = B.
template <int DK>
__global__ void __launch_bounds__(GD_THREADS, gd_blocks(DK)) gated_delta_step_kernel(const DeltaParams p)
{
    extern __shared__ __align__(16) float gd_smem[];
    const int col0 = blockIdx.x * GD_COLS, hv = blockIdx.y, b = blockIdx.z;
    const int i = threadIdx.x & 3, col = threadIdx.x >> 2;
    const int cap = max(p.T, p.prev_T);
    const GdSmem<DK> sm(gd_smem, cap);
    pdl_launch_dependents();
    pdl_wait_prior();
    // rows, which need no slot, are asked for before it is waited for
    const DeltaRows &lead = p.prev_T > 0 ? p.prev : p.rows;
    const int lead_T = p.prev_T > 0 ? p.prev_T : p.T;
    const int slot = p.state_idx ? p.state_idx[b] : b;
    const int accept = p.accept_len && p.prev_T > 0 ? p.accept_len[b] : p.prev_T;
    GdFirst<DK> f;
    gd_first<DK>(p, lead, static_cast<long long>(b) * lead_T, lead_T, hv, col0, p.prev_T == 0, f);
    uint16_t *o = p.o + static_cast<long long>(b) * p.T * p.ldo + static_cast<long long>(hv) * p.dv + col0;
    if (slot < 0 || slot >= p.n_slots) {        // an inactive entry: its outputs are zero
        if (slot >= 0 && threadIdx.x == 0) atomicOr(p.err, 8);
        for (int t = 0; t < p.T; ++t)
            if (i == 0) o[t * p.ldo + col] = 0;
        return;
    }
    float *s = p.state + ((static_cast<long long>(slot) * p.Hv + hv) * p.dv + col0 + col) * DK;
    GdState<DK> st;
    st.load(s, i);
    if (p.prev_T > 0) {
        const int n = p.accept_len ? min(p.prev_T, max(0, min(accept, p.prev_T) + 1)) : p.prev_T;
        if (n > 0) {
            const bool running = gd_stage<DK>(p, p.prev, static_cast<long long>(b) * p.prev_T, n, hv, col0, sm, false, f);
            gd_rows<DK, false>(st, sm, n, running, nullptr, 0);
            if (!p.commit) st.store(s, i);
            __syncthreads();
        }
        if (p.T > 0) gd_first<DK>(p, p.rows, static_cast<long long>(b) * p.T, p.T, hv, col0, true, f);
    }
    if (p.T > 0) {
        const bool running = gd_stage<DK>(p, p.rows, static_cast<long long>(b) * p.T, p.T, hv, col0, sm, true, f);
        gd_rows<DK, true>(st, sm, p.T, running, o, p.ldo);
    }
    if (p.commit) st.store(s, i);
}

// ------------------------------------------------ several rows at once
//
// With a few rows the state need not be walked row by row.  Let n rows (the
// accepted ones of prev, then the new ones) have running log decays G and
// inverse norms r_k, r_q.  From the state S before all of them
//   r_t = beta_t (v_t - e^(G_t) r_k,t (S k_t))
//   u_t = r_t - sum_{s<t} A_ts u_s,  A_ts = beta_t e^(G_t - G_s) r_k,t r_k,s (k_t . k_s)
//   o_t = scale e^(G_t) r_q,t (S q_t) + sum_{s<=t} M_ts u_s,
//         M_ts = scale e^(G_t - G_s) r_q,t r_k,s (q_t . k_s)
//   S'  = e^(G_m) S + sum_{s<m} (e^(G_m - G_s) r_k,s u_s) k_s^T
// where the state is wanted after the first m rows: the accepted ones, or all.
//
// A warp owns 16 rows of S, or half the columns of 16 rows (KS = 2: the two
// warps' parts of S k and S q meet in shared memory, and both go on).  S k and
// S q are tf32 products with S as the A operand, in two terms (22 bits; keys
// and queries, bf16 as they come, are exact in tf32), and so is the update,
// with u in two terms and S as the accumulator.  Everything between is fp32.
// The block computes A and M once for its warps.  Up to 16 rows in all, r, u
// and the outputs stay in the products' accumulator layout: one pass over the
// rows hands each u to the other lanes, which subtract it from their r and add
// it to their o.  With more rows u comes by substitution in shared memory.
//
// A block has 64 state rows; a warp copies its rows to shared memory while the
// chain of small steps (gates, norms, A) runs, and back through it (8-byte
// stores from the accumulators take 10 us more at 256 x (4 + 4) rows).
//
// A NaN or an infinity in a row reaches that row and later ones only.
//
// Measured, 48 heads of 128 x 128: 256 sequences with 4 rows and 4 replayed
// 242 us, 6.9 TB/s, HBM-bound (five blocks a multiprocessor); with 8 and 8,
// 320 us (four).  4 sequences with 8 and 8 rows 9.7 us (10.5 with one warp for
// 16 state rows), of which 3.9 are traffic: the chain of a block -- slot and
// gates from memory, running sum, decays, A, S k, u, update -- takes 5.4 us by
// itself (one sequence).

constexpr int GB_KPAD = 8, GB_FPAD = 4;         // padding of a row in shared memory, bf16 and fp32 values

// v as two tf32 terms, 22 bits of it; the second's low bits are not read.
__device__ __forceinline__ void gb_split_tf32(float v, uint32_t &hi, uint32_t &lo)
{
    hi = __float_as_uint(v) & 0xFFFFE000u;
    lo = __float_as_uint(v - __uint_as_float(hi));
}

// Sums of two floats each, kept as the rounded sum and what it leaves:
// differences of large sums give the decays between near rows.
struct Sum2 {
    float hi, lo;
};

__device__ __forceinline__ Sum2 add2(Sum2 a, Sum2 b)
{
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float hi = s + e;
    return Sum2{hi, e - (hi - s)};
}

__device__ __forceinline__ float exp_diff(Sum2 a, float bhi, float blo) { return expf((a.hi - bhi) + (a.lo - blo)); }

constexpr int GB_COLS = 64;                     // state rows of a block
constexpr int gb_threads(int KS) { return 2 * GB_COLS * KS; }  // KS warps for 16 of them, a part of the columns each

// Shared memory of a block: NP rows in all, NQR new ones (8 or multiples of 16).
template <int DK, int NP, int NQR, int KS>
struct GbSmem {
    static constexpr bool SMALL = NP <= 16;     // r, u and o stay in registers
    float s[GB_COLS][DK + 8];                   // the state (rows padded: fragment loads free of bank conflicts)
    uint16_t k[NP][DK + GB_KPAD], q[NQR][DK + GB_KPAD], v[NP][GB_COLS + GB_KPAD];
    float a[NP][NP + GB_FPAD];                  // A, [t][s]; SMALL: [s][t]
    float m[SMALL ? NP : NQR][(SMALL ? NQR : NP) + GB_FPAD];    // M, [t][s]; SMALL: [s][t]
    float u[SMALL ? 1 : GB_COLS][NP + GB_FPAD];
    float ed[SMALL ? NP : 1][NP + GB_FPAD];     // decays between rows
    float g_hi[NP], g_lo[NP], beta[NP], rk[NP], rq[NQR], f_p[NP], f_s[NP], f_o;
    float part[KS == 1 ? 1 : 4 * KS][(NP + NQR) / 2][32];   // KS > 1: the warps' parts of S k and S q
};

// D (16x8 fp32) += A (16x8 tf32, row) * B (8x8 tf32, col); the operands' low 13 bits are not read.
__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NK, NQ: most n8 tiles of rows and of new rows.  Grid: x = dv / GB_COLS,
// y = Hv, z = B.
template <int DK, int NK, int NQ, int KS>
__global__ void __launch_bounds__(gb_threads(KS), 4 / KS) gated_delta_block_kernel(const DeltaParams p)
{
    extern __shared__ __align__(16) uint8_t gb_smem[];
    constexpr int NP = 8 * NK, NQR = 8 * NQ;
    using Smem = GbSmem<DK, NP, NQR, KS>;
    constexpr bool SMALL = Smem::SMALL;
    Smem &sm = *reinterpret_cast<Smem *>(gb_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    constexpr int THREADS = gb_threads(KS), NWARP = THREADS / 32, COLS = DK / KS;
    static_assert(KS == 1 || SMALL, "the parts meet in the accumulator layout");
    const int wr = warp & 3, wk = warp >> 2;    // 16 state rows, COLS columns
    const int col0 = blockIdx.x * GB_COLS, hv = blockIdx.y, b = blockIdx.z, hk = hv / (p.Hv / p.Hk);
    pdl_launch_dependents();
    pdl_wait_prior();
    int na = p.prev_T;                          // accepted rows
    const int accept = p.accept_len && na > 0 ? p.accept_len[b] : na;
    const int slot = gd_slot(p.state_idx, p.n_slots, b, p.err);
    uint16_t *o = p.o + static_cast<long long>(b) * p.T * p.ldo + static_cast<long long>(hv) * p.dv + col0;
    if (slot < 0) {                             // an inactive entry: its outputs are zero
        for (int i = tid; i < p.T * GB_COLS; i += THREADS) o[(i / GB_COLS) * p.ldo + i % GB_COLS] = 0;
        return;
    }
    float *state = p.state + ((static_cast<long long>(slot) * p.Hv + hv) * p.dv + col0) * DK;
    if (na > 0) na = min(na, max(0, min(accept, na) + 1));
    const int rows = na + p.T, tn = (p.T + 7) >> 3, nk = (rows + 7) >> 3;
    const int kept = p.commit ? rows : na;      // rows that the state is wanted after
    const long long pr0 = static_cast<long long>(b) * p.prev_T, nr0 = static_cast<long long>(b) * p.T;

    // gates of two rows a lane, for the last warp; asked for first, as the
    // chain of small steps that the block waits for begins with them
    const bool gate_warp = warp == NWARP - 1;
    float gate[2] = {0.f, 0.f}, rate[2] = {0.f, 0.f};
    if (gate_warp)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            if (t < na) {
                gate[e] = p.prev.g[(pr0 + t) * p.prev.ldg + hv];
                rate[e] = p.prev.beta[(pr0 + t) * p.prev.ldg + hv];
            } else if (t < rows) {
                gate[e] = p.rows.g[(nr0 + t - na) * p.rows.ldg + hv];
                rate[e] = p.rows.beta[(nr0 + t - na) * p.rows.ldg + hv];
            }
        }
    // ---- rows into shared memory as they are; absent rows are zero
    {
        constexpr int PR = DK / 8, PV = GB_COLS / 8;    // 16-byte pieces of a key row, of a value row
        auto piece = [&](uint16_t *dst, const uint16_t *src, bool live) {
            if (live)
                cp_async_16(smem_addr(dst), src);
            else
                *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
        };
        const int jk = tid % PR * 8, jv = tid % PV * 8;
        const uint16_t *k_old = p.prev.k + pr0 * p.prev.ldk + hk * DK + jk, *k_new = p.rows.k + (nr0 - na) * p.rows.ldk + hk * DK + jk;
        const uint16_t *v_old = p.prev.v + pr0 * p.prev.ldv + hv * p.dv + col0 + jv,
                       *v_new = p.rows.v + (nr0 - na) * p.rows.ldv + hv * p.dv + col0 + jv;
        const uint16_t *q_new = p.rows.q + nr0 * p.rows.ldq + hk * DK + jk;
#pragma unroll
        for (int t0 = 0; t0 < NP; t0 += THREADS / PR)
            if (const int t = t0 + tid / PR; t < NP) piece(&sm.k[t][jk], t < na ? k_old + t * p.prev.ldk : k_new + t * p.rows.ldk, t < rows);
#pragma unroll
        for (int t0 = 0; t0 < NQR; t0 += THREADS / PR)
            if (const int t = t0 + tid / PR; t < NQR) piece(&sm.q[t][jk], q_new + t * p.rows.ldq, t < p.T);
#pragma unroll
        for (int t0 = 0; t0 < NP; t0 += THREADS / PV)
            if (const int t = t0 + tid / PV; t < NP) piece(&sm.v[t][jv], t < na ? v_old + t * p.prev.ldv : v_new + t * p.rows.ldv, t < rows);
    }
    cp_async_commit();
    // ---- the warp's state rows
    float *srows = state + 16 * wr * DK + wk * COLS;
#pragma unroll 4
    for (int i = lane; i < 16 * COLS / 4; i += 32) {
        const int r = i / (COLS / 4), j = i % (COLS / 4) * 4;
        cp_async_16(smem_addr(&sm.s[16 * wr + r][wk * COLS + j]), srows + r * DK + j);
    }
    cp_async_commit();
    if (gate_warp) {
        // the running sum of the log decays
        Sum2 G[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            G[e] = Sum2{gate[e] < GD_MIN_LOG ? GD_MIN_LOG : gate[e], 0.f};
        }
        Sum2 run = add2(G[0], G[1]);
#pragma unroll 1
        for (int d = 1; d < 4 * NK; d <<= 1) {
            const Sum2 below{__shfl_up_sync(0xFFFFFFFFu, run.hi, d), __shfl_up_sync(0xFFFFFFFFu, run.lo, d)};
            if (lane >= d) run = add2(below, run);
        }
        Sum2 before{__shfl_up_sync(0xFFFFFFFFu, run.hi, 1), __shfl_up_sync(0xFFFFFFFFu, run.lo, 1)};
        if (lane == 0) before = Sum2{0.f, 0.f};
        G[0] = add2(before, G[0]);
        G[1] = run;
        if (2 * lane < NP)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sm.g_hi[2 * lane + e] = G[e].hi;
                sm.g_lo[2 * lane + e] = G[e].lo;
                sm.beta[2 * lane + e] = rate[e];
            }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");        // the rows; the state may take longer
    __syncthreads();
    // ---- decays: up to each row, from it to the last kept one, between rows
    if (gate_warp) {
        const float mh = kept > 0 ? sm.g_hi[kept - 1] : 0.f, ml = kept > 0 ? sm.g_lo[kept - 1] : 0.f;
#pragma unroll 1
        for (int t = lane; t < NP; t += 32) {
            const float hi = sm.g_hi[t], lo = sm.g_lo[t];
            sm.f_p[t] = expf(hi + lo);
            sm.f_s[t] = t < kept ? expf((mh - hi) + (ml - lo)) : 0.f;
        }
        if (lane == 0) sm.f_o = expf(mh + ml);
    }
    // ---- inverse norms, four lanes a row
#pragma unroll 1
    for (int t = tid >> 2; t < NP + NQR; t += THREADS / 4) {
        const uint16_t *row = t >= NP ? sm.q[t - NP] : sm.k[t];
        float ss[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < DK / 32; ++j) {
            const uint4 u = *reinterpret_cast<const uint4 *>(row + 32 * j + 8 * c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
                ss[0] = fmaf(lo, lo, ss[0]);
                ss[1] = fmaf(hi, hi, ss[1]);
            }
        }
        ss[0] += ss[1];
        // the lanes of a row are together in its loop (NP + NQR is a multiple of 8 rows, a warp's part of it)
        ss[0] += __shfl_xor_sync(0xFFFFFFFFu, ss[0], 1);
        ss[0] += __shfl_xor_sync(0xFFFFFFFFu, ss[0], 2);
        const float inv = p.l2norm ? rsqrtf(ss[0] + GD_L2_EPS) : 1.f;
        if (c == 0) {
            if (t >= NP)
                sm.rq[t - NP] = inv * p.scale;
            else
                sm.rk[t] = inv;
        }
    }
    if constexpr (SMALL) {
#pragma unroll
        for (int i0 = 0; i0 < NP * NP; i0 += THREADS) {
            const int i = i0 + tid, t = i / NP, s = i % NP;
            if (i < NP * NP) sm.ed[t][s] = s <= t ? exp_diff(Sum2{sm.g_hi[t], sm.g_lo[t]}, sm.g_hi[s], sm.g_lo[s]) : 0.f;
        }
    }
    __syncthreads();

    // ---- A and M, by tiles of 16 rows and 8 columns
    constexpr int AT = (NP + 15) / 16, MT = (NQR + 15) / 16;
#pragma unroll 1
    for (int task = warp; task < (AT + MT) * NK; task += NWARP) {
        const int j = task % NK, row_tile = task / NK;
        const bool is_m = row_tile >= AT;
        const int mt = is_m ? row_tile - AT : row_tile;
        const int r0 = is_m ? na + 16 * mt : 16 * mt;           // the tile's first row among all
        if (is_m ? 16 * mt >= p.T : r0 >= rows) continue;
        float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        // eight rows fill half a tile: the other half repeats them
        const uint16_t *arow = (is_m ? sm.q[16 * mt + (lane & (NQR < 16 ? 7 : 15))] : sm.k[16 * mt + (lane & (NP < 16 ? 7 : 15))]) + (lane >> 4) * 8;
        if (8 * j <= r0 + 15) {
#pragma unroll
            for (int s = 0; s < DK / 32; ++s) {
                uint32_t a0[4], a1[4], bb[4];
                ldmatrix_x4(a0, smem_addr(arow + 32 * s));
                ldmatrix_x4(a1, smem_addr(arow + 32 * s + 16));
                ldmatrix_x4(bb, smem_addr(sm.k[8 * j + (lane & 7)] + 32 * s + (lane >> 3) * 8));
                mma_bf16_16816(acc[0], a0[0], a0[1], a0[2], a0[3], bb[0], bb[1]);
                mma_bf16_16816(acc[1], a1[0], a1[1], a1[2], a1[3], bb[2], bb[3]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tl = 16 * mt + g + 8 * h, t = r0 + g + 8 * h;     // within its matrix, among all rows
            const bool live = is_m ? tl < p.T : t < rows;
            if (tl >= (is_m ? NQR : NP)) continue;
            const Sum2 G = live ? Sum2{sm.g_hi[t], sm.g_lo[t]} : Sum2{0.f, 0.f};
            const float f = !live ? 0.f : is_m ? sm.rq[tl] : sm.beta[t] * sm.rk[t];
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int s = 8 * j + 2 * c + e;
                const float d = !live || s > t ? 0.f : SMALL ? sm.ed[SMALL ? t : 0][s] : exp_diff(G, sm.g_hi[s], sm.g_lo[s]);
                v[e] = live && (is_m ? s <= t : s < t) ? (acc[0][2 * h + e] + acc[1][2 * h + e]) * (d * sm.rk[s] * f) : 0.f;
            }
            const int s0 = 8 * j + 2 * c;
            if constexpr (SMALL) {
                (is_m ? sm.m[s0] : sm.a[s0])[tl] = v[0];
                (is_m ? sm.m[s0 + 1] : sm.a[s0 + 1])[tl] = v[1];
            } else {
                *reinterpret_cast<float2 *>(is_m ? &sm.m[tl][s0] : &sm.a[tl][s0]) = make_float2(v[0], v[1]);
            }
        }
    }

    // ---- S k and S q
    float pk[NK][4], pq[NQ][4];
    float lk[SMALL ? NK : 1][4] = {}, lq[4] = {};   // SMALL: the second terms' sums, to halve the chains of products
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) pk[j][e] = 0.f;
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) pq[j][e] = 0.f;
    cp_async_wait_all();
    __syncwarp();                               // the warp's state rows are in
    float *srow = &sm.s[16 * wr + g][wk * COLS + 2 * c];
    constexpr int SST = DK + 8;
#pragma unroll 4
    for (int s = 0; s < COLS / 8; ++s) {
        // columns 2 c and 2 c + 1 of the step are its k = c and c + 4
        const float2 x = *reinterpret_cast<const float2 *>(srow + 8 * s), y = *reinterpret_cast<const float2 *>(srow + 8 * SST + 8 * s);
        const float sv[4] = {x.x, y.x, x.y, y.y};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) gb_split_tf32(sv[i], hi[i], lo[i]);
        auto product = [&](float (&d)[4], float (&d_lo)[4], const uint16_t *row) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(row + wk * COLS + 8 * s + 2 * c);
            const uint32_t b0 = w << 16, b1 = w & 0xFFFF0000u;
            mma_tf32_1688(d_lo, lo[0], lo[1], lo[2], lo[3], b0, b1);
            mma_tf32_1688(d, hi[0], hi[1], hi[2], hi[3], b0, b1);
        };
#pragma unroll
        for (int j = 0; j < NK; ++j)
            if (j < nk) product(pk[j], SMALL ? lk[SMALL ? j : 0] : pk[j], sm.k[8 * j + g]);
#pragma unroll
        for (int j = 0; j < NQ; ++j)
            if (j < tn) product(pq[j], SMALL ? lq : pq[j], sm.q[8 * j + g]);
    }
    if constexpr (SMALL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int j = 0; j < NK; ++j) pk[j][e] += lk[j][e];
            pq[0][e] += lq[e];
        }
    }
    const int nu = (kept + 7) >> 3;
    if constexpr (KS > 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int j = 0; j < NK; ++j) sm.part[warp][4 * j + e][lane] = pk[j][e];
#pragma unroll
            for (int j = 0; j < NQ; ++j) sm.part[warp][4 * (NK + j) + e][lane] = pq[j][e];
        }
    }
    __syncthreads();                            // A and M are complete, and the parts
    if constexpr (KS > 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int j = 0; j < NK; ++j) pk[j][e] = sm.part[wr][4 * j + e][lane] + sm.part[wr + 4][4 * j + e][lane];
#pragma unroll
            for (int j = 0; j < NQ; ++j) pq[j][e] = sm.part[wr][4 * (NK + j) + e][lane] + sm.part[wr + 4][4 * (NK + j) + e][lane];
        }
    }
    // ---- r
#pragma unroll
    for (int j = 0; j < NK; ++j)
        if (j < nk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 8 * j + 2 * c + (e & 1);
                pk[j][e] = sm.beta[t] * (bf16_bits_to_float(sm.v[t][16 * wr + g + 8 * (e >> 1)]) - sm.f_p[t] * sm.rk[t] * pk[j][e]);
            }
    if constexpr (SMALL) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 8 * j + 2 * c + (e & 1);
                pq[j][e] = t < p.T ? sm.f_p[na + t] * sm.rq[t] * pq[j][e] : 0.f;
            }
        // row s's u, complete once the rows before it have been taken off its
        // r, goes to the lanes of its state rows
#pragma unroll
        for (int s = 0; s < 8 * NK; ++s) {
            if (s >= rows) break;
            const int from = (lane & ~3) | ((s & 7) >> 1);
            const float ug = __shfl_sync(0xFFFFFFFFu, pk[s >> 3][s & 1], from), uh = __shfl_sync(0xFFFFFFFFu, pk[s >> 3][2 + (s & 1)], from);
#pragma unroll
            for (int j = s >> 3; j < NK; ++j) {
                const float2 av = *reinterpret_cast<const float2 *>(&sm.a[s][8 * j + 2 * c]);
                const bool on0 = 8 * j + 2 * c > s, on1 = 8 * j + 2 * c + 1 > s;   // (a NaN stays with later rows)
                if (on0) pk[j][0] = fmaf(-av.x, ug, pk[j][0]);
                if (on1) pk[j][1] = fmaf(-av.y, ug, pk[j][1]);
                if (on0) pk[j][2] = fmaf(-av.x, uh, pk[j][2]);
                if (on1) pk[j][3] = fmaf(-av.y, uh, pk[j][3]);
            }
            if (tn > 0)
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const float2 mv = *reinterpret_cast<const float2 *>(&sm.m[SMALL ? s : 0][8 * j + 2 * c]);
                    const bool on0 = na + 8 * j + 2 * c >= s, on1 = na + 8 * j + 2 * c + 1 >= s;
                    if (on0) pq[j][0] = fmaf(mv.x, ug, pq[j][0]);
                    if (on1) pq[j][1] = fmaf(mv.y, ug, pq[j][1]);
                    if (on0) pq[j][2] = fmaf(mv.x, uh, pq[j][2]);
                    if (on1) pq[j][3] = fmaf(mv.y, uh, pq[j][3]);
                }
        }
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 8 * j + 2 * c + (e & 1);
                if (wk == 0 && t < p.T) o[t * p.ldo + 16 * wr + g + 8 * (e >> 1)] = __bfloat16_as_ushort(__float2bfloat16_rn(pq[j][e]));
            }
    } else {
        // u by forward substitution in the warp's own rows of shared memory, a
        // state row a lane, eight rows t at a time
        float (*uw)[NP + GB_FPAD] = &sm.u[16 * wr];
#pragma unroll
        for (int j = 0; j < NK; ++j)
            if (j < nk)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(&uw[g + 8 * h][8 * j + 2 * c]) = make_float2(pk[j][2 * h], pk[j][2 * h + 1]);
        __syncwarp();
        if (lane < 16) {
            float *ur = uw[lane];
#pragma unroll 1
            for (int j = 0; j < nk; ++j) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(ur + 8 * j + i);
                    u[i] = x.x;
                    u[i + 1] = x.y;
                    u[i + 2] = x.z;
                    u[i + 3] = x.w;
                }
#pragma unroll 1
                for (int k = 0; k < 2 * j; ++k) {   // four earlier rows
                    const float4 e = *reinterpret_cast<const float4 *>(ur + 4 * k);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 av = *reinterpret_cast<const float4 *>(&sm.a[8 * j + i][4 * k]);
                        u[i] -= (av.x * e.x + av.y * e.y) + (av.z * e.z + av.w * e.w);
                    }
                }
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    const float4 a1 = *reinterpret_cast<const float4 *>(&sm.a[8 * j + i][8 * j]);
                    const float4 a2 = *reinterpret_cast<const float4 *>(&sm.a[8 * j + i][8 * j + 4]);
                    const float av[8] = {a1.x, a1.y, a1.z, a1.w, a2.x, a2.y, a2.z, a2.w};
#pragma unroll
                    for (int k = 0; k < i; ++k) u[i] = fmaf(-av[k], u[k], u[i]);
                }
                *reinterpret_cast<float4 *>(ur + 8 * j) = make_float4(u[0], u[1], u[2], u[3]);
                *reinterpret_cast<float4 *>(ur + 8 * j + 4) = make_float4(u[4], u[5], u[6], u[7]);
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NQ; ++j)
            if (j < tn) {
                const int t0 = 8 * j + 2 * c;
                float s[4];                     // (t0, g) (t0 + 1, g) (t0, g + 8) (t0 + 1, g + 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = (t0 + (e & 1) < p.T ? sm.f_p[na + t0 + (e & 1)] * sm.rq[t0 + (e & 1)] : 0.f) * pq[j][e];
#pragma unroll 1
                for (int k = 0; k < min(na + 8 * j + 8, 8 * nk); k += 4) {
                    const float4 m0 = *reinterpret_cast<const float4 *>(&sm.m[SMALL ? 0 : t0][k]), m1 = *reinterpret_cast<const float4 *>(&sm.m[SMALL ? 0 : t0 + 1][k]);
                    const float4 u0 = *reinterpret_cast<const float4 *>(&uw[g][k]), u1 = *reinterpret_cast<const float4 *>(&uw[g + 8][k]);
                    const float ma[4] = {m0.x, m0.y, m0.z, m0.w}, mb[4] = {m1.x, m1.y, m1.z, m1.w};
                    const float ua[4] = {u0.x, u0.y, u0.z, u0.w}, ub[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool on0 = na + t0 >= k + i, on1 = na + t0 + 1 >= k + i;   // (a NaN stays with later rows)
                        if (on0) s[0] = fmaf(ma[i], ua[i], s[0]);
                        if (on1) s[1] = fmaf(mb[i], ua[i], s[1]);
                        if (on0) s[2] = fmaf(ma[i], ub[i], s[2]);
                        if (on1) s[3] = fmaf(mb[i], ub[i], s[3]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + (e & 1) < p.T)
                        o[(t0 + (e & 1)) * p.ldo + 16 * wr + g + 8 * (e >> 1)] = __bfloat16_as_ushort(__float2bfloat16_rn(s[e]));
            }
    }
    // ---- the state after the wanted rows: S <- decay S + u' K, u' = u f_s r_k in two terms
    if (nu == 0) return;
    const float decay = sm.f_o;
    uint32_t uh[2][4], ul[2][4];
    auto scaled_u = [&](int j, float x0, float x1, float y0, float y1, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
        const int t = 8 * j + 2 * c;            // rows t, t + 1 of state row g (x) and g + 8 (y): the products' k = c and c + 4
        const float w0 = sm.f_s[t] * sm.rk[t], w1 = sm.f_s[t + 1] * sm.rk[t + 1];
        const bool in0 = t < kept, in1 = t + 1 < kept;
        const float v[4] = {in0 ? x0 * w0 : 0.f, in0 ? y0 * w0 : 0.f, in1 ? x1 * w1 : 0.f, in1 ? y1 * w1 : 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) gb_split_tf32(v[e], hi[e], lo[e]);
    };
    if constexpr (SMALL)
#pragma unroll
        for (int j = 0; j < NK; ++j)
            if (j < nu) scaled_u(j, pk[j][0], pk[j][1], pk[j][2], pk[j][3], uh[SMALL ? j : 0], ul[SMALL ? j : 0]);
#pragma unroll 1
    for (int i = 0; i < COLS / 32; ++i) {
        float st[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = *reinterpret_cast<const float2 *>(srow + 32 * i + 8 * e), y = *reinterpret_cast<const float2 *>(srow + 8 * SST + 32 * i + 8 * e);
            st[e][0] = decay * x.x;
            st[e][1] = decay * x.y;
            st[e][2] = decay * y.x;
            st[e][3] = decay * y.y;
        }
        auto add = [&](int j, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
            uint32_t bb[4];
            ldmatrix_x4_trans(bb, smem_addr(sm.k[8 * j + (lane & 7)] + wk * COLS + 32 * i + (lane >> 3) * 8));
            // rows 8 j + 2 c and + 1, zero where not kept: their u is, but a key may hold a NaN
            const int t = 8 * j + 2 * c;
            const uint32_t rows_in = t + 1 < kept ? 0xFFFFFFFFu : t < kept ? 0xFFFFu : 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t b = bb[e] & rows_in, b0 = b << 16, b1 = b & 0xFFFF0000u;
                mma_tf32_1688(st[e], lo[0], lo[1], lo[2], lo[3], b0, b1);
                mma_tf32_1688(st[e], hi[0], hi[1], hi[2], hi[3], b0, b1);
            }
        };
        if constexpr (SMALL) {
#pragma unroll
            for (int j = 0; j < NK; ++j)
                if (j < nu) add(j, uh[SMALL ? j : 0], ul[SMALL ? j : 0]);
        } else {
#pragma unroll 1
            for (int j = 0; j < nu; ++j) {
                const float2 x = *reinterpret_cast<const float2 *>(&sm.u[SMALL ? 0 : 16 * wr + g][8 * j + 2 * c]),
                             y = *reinterpret_cast<const float2 *>(&sm.u[SMALL ? 0 : 16 * wr + g + 8][8 * j + 2 * c]);
                scaled_u(j, x.x, x.y, y.x, y.y, uh[0], ul[0]);
                add(j, uh[0], ul[0]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            *reinterpret_cast<float2 *>(srow + 32 * i + 8 * e) = make_float2(st[e][0], st[e][1]);
            *reinterpret_cast<float2 *>(srow + 8 * SST + 32 * i + 8 * e) = make_float2(st[e][2], st[e][3]);
        }
    }
    __syncwarp();
#pragma unroll 4
    for (int i = lane; i < 16 * COLS / 4; i += 32) {
        const int r = i / (COLS / 4), j = i % (COLS / 4) * 4;
        *reinterpret_cast<float4 *>(srows + r * DK + j) = *reinterpret_cast<const float4 *>(&sm.s[16 * wr + r][wk * COLS + j]);
    }
}

}  // namespace sv
