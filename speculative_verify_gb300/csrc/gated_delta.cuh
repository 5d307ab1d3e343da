// gated_delta.cuh -- the gated delta rule row by row, for decode and verify
// rows.
//
// Each value head keeps a state S of dv rows and dk columns (fp32).  A row
// with key k, query q, value v, log decay g and rate beta does
//
//   S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q
//
// The dv rows of S never mix, so a block takes `cols` of them of one head of
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
constexpr float GD_MAX_LOG = 10.f;              // largest |sum of log decays| kept outside the state
constexpr float GD_L2_EPS = 1e-6f;

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
    int cols;                                   // state rows of a block, blockDim.x / 4
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
// [GD][cols], then per row beta, e^g, the running decay, its inverse, q.k.
__host__ __device__ constexpr int gd_smem_floats(int rows, int dk, int cols) { return rows * (2 * dk + cols + 5); }

template <int DK>
struct GdSmem {
    float *k, *q, *v, *beta, *eg, *c, *cinv, *qk;
    __device__ __forceinline__ GdSmem(float *base, int rows, int cols)
    {
        k = base;
        q = k + rows * DK;
        v = q + rows * DK;
        beta = v + rows * cols;
        eg = beta + rows;
        c = eg + rows;
        cinv = c + rows;
        qk = cinv + rows;
    }
};

// Stage `n` rows (first row r0) of head hv in shared memory: keys and queries
// in fp32 (normalised where asked, the query times `scale`), q.k, this
// block's values, the gates and their running products.  Returns whether the
// running products may be used (uniform over the block).
template <int DK>
__device__ __forceinline__ bool gd_stage(const DeltaParams &p, const DeltaRows &r, long long r0, int n, int hv, int col0,
                                         int cols, const GdSmem<DK> &sm, bool want_q)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
    constexpr int E = DK / 32;                  // a lane's values of a row, consecutive
    const int hk = hv / (p.Hv / p.Hk);
    for (int t = warp; t < n; t += nwarp) {
        float k[E], q[E];
        float kk = 0.f, qq = 0.f, qk = 0.f;
        auto load = [&](const uint16_t *src, float (&d)[E]) {
            if constexpr (E == 4) {
                const uint2 u = *reinterpret_cast<const uint2 *>(src + lane * E);
                d[0] = __uint_as_float(u.x << 16);
                d[1] = __uint_as_float(u.x & 0xFFFF0000u);
                d[2] = __uint_as_float(u.y << 16);
                d[3] = __uint_as_float(u.y & 0xFFFF0000u);
            } else {
                const uint32_t u = *reinterpret_cast<const uint32_t *>(src + lane * E);
                d[0] = __uint_as_float(u << 16);
                d[1] = __uint_as_float(u & 0xFFFF0000u);
            }
        };
        load(r.k + (r0 + t) * r.ldk + static_cast<long long>(hk) * DK, k);
        if (want_q) {
            load(r.q + (r0 + t) * r.ldq + static_cast<long long>(hk) * DK, q);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) q[e] = 0.f;
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
    // values: eight per thread (cols is a multiple of 32)
    for (int i = tid; i < n * (cols / 8); i += blockDim.x) {
        const int t = i / (cols / 8), j = (i - t * (cols / 8)) * 8;
        const uint4 u = *reinterpret_cast<const uint4 *>(r.v + (r0 + t) * r.ldv + static_cast<long long>(hv) * p.dv + col0 + j);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sm.v[t * cols + j + 2 * e] = __uint_as_float(w[e] << 16);
            sm.v[t * cols + j + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    // gates; the running sum of the log decays by a warp scan (n <= 32)
    bool ok = true;
    if (warp == 0) {
        const float g = lane < n ? r.g[(r0 + lane) * r.ldg + hv] : 0.f;
        float G = g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float below = __shfl_up_sync(0xFFFFFFFFu, G, o);
            if (lane >= o) G += below;
        }
        ok = fabsf(G) <= GD_MAX_LOG;            // false for a NaN too
        if (lane < n) {
            sm.beta[lane] = r.beta[(r0 + lane) * r.ldg + hv];
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
__device__ __forceinline__ void gd_rows(GdState<DK> &st, const GdSmem<DK> &sm, int n, int cols, bool running,
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
        const float u = sm.beta[t] * (sm.v[t * cols + col] - c * a);
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

// Grid: x = dv / cols, y = Hv, z = B.
template <int DK>
__global__ void __launch_bounds__(512) gated_delta_step_kernel(const DeltaParams p)
{
    extern __shared__ __align__(16) float gd_smem[];
    const int cols = p.cols, col0 = blockIdx.x * cols, hv = blockIdx.y, b = blockIdx.z;
    const int i = threadIdx.x & 3, col = threadIdx.x >> 2;
    const int cap = max(p.T, p.prev_T);
    const GdSmem<DK> sm(gd_smem, cap, cols);
    pdl_launch_dependents();
    pdl_wait_prior();
    uint16_t *o = p.o + static_cast<long long>(b) * p.T * p.ldo + static_cast<long long>(hv) * p.dv + col0;
    const int slot = gd_slot(p.state_idx, p.n_slots, b, p.err);
    if (slot < 0) {                             // an inactive entry: its outputs are zero
        for (int t = 0; t < p.T; ++t)
            if (i == 0) o[t * p.ldo + col] = 0;
        return;
    }
    float *s = p.state + ((static_cast<long long>(slot) * p.Hv + hv) * p.dv + col0 + col) * DK;
    GdState<DK> st;
    st.load(s, i);
    int n = p.prev_T;
    if (p.accept_len && n > 0) n = min(n, max(0, min(p.accept_len[b], n) + 1));
    if (n > 0) {
        const bool running = gd_stage<DK>(p, p.prev, static_cast<long long>(b) * p.prev_T, n, hv, col0, cols, sm, false);
        gd_rows<DK, false>(st, sm, n, cols, running, nullptr, 0);
        if (!p.commit) st.store(s, i);
        __syncthreads();
    }
    if (p.T > 0) {
        const bool running = gd_stage<DK>(p, p.rows, static_cast<long long>(b) * p.T, p.T, hv, col0, cols, sm, true);
        gd_rows<DK, true>(st, sm, p.T, cols, running, o, p.ldo);
    }
    if (p.commit) st.store(s, i);
}

}  // namespace sv
