// kv4_attn.cuh -- attention of a few query rows over the 4-bit cache, straight
// from the packed pages on mma.sync: o = softmax(scale q k^T) v, row by row
// over the tokens that it sees.
//
// A warp takes a page of its head's item (kv4_plan.cuh) at a time, from a ring
// of its own filled by bulk copies, and keeps a running softmax of its own; the
// warps of a block join at the item's end.  Products are m16n8k16 of fp16, with
// the cache as the operand of 16 rows: scores^T = K Q^T and o^T = V^T P^T, NQ
// times 8 packed query rows (with queries as the 16 rows, half of the products
// and of the softmax are of rows that are not there).  Keys and values become
// fp16 in registers, exactly (kv4.cuh): one conversion and one product a pair.
//   * Scores: a thread's A rows are two tokens and its K steps are a token's 32
//     neighbouring dimensions, so a token's codes come in one 16-byte load.
//     Queries are laid out the same, times a power of two of their row that
//     puts the largest in [2^14, 2^15): exact but for values 2^-25 of it.
//   * Values: probabilities, transposed in registers (movmatrix), are the B
//     operand; an A row is a dimension, and a pair of tokens' values are put
//     together by byte permutation.  Thread row g has dimensions g d / 8 .., so
//     that it ends with neighbouring ones.
//   * Sums and the softmax are fp32, probabilities fp16 (where 8 bits of bf16
//     would show in the outputs).  They are taken relative to 2^-7 of a maximum
//     that is only moved when a score passes it by 2^8, so most pages rescale
//     nothing and fp16's range is used up to 2^15: each is off by 2^-11 of itself
//     at most, or by 2^-32 of the largest where that is more.  Relative to the
//     maximum it is 2^-25, and their sum has the unrounded ones: of 131,072 tokens
//     at 2^-25.2 of the largest, 0.3 % of the weight, nothing reached the outputs.
//
// Bound by instructions, not by HBM: about 680 a warp and page of d 128, most
// of them conversions and the products and permutations that go with them.
// 256 rows of 4,096 tokens (32 query heads, 8 of 128) take 184 us, 5.0 TB/s;
// 64 x 4 rows in a window of 4,096 (16 query heads, 8 of 64) 52 us, 2.9 TB/s,
// a page there being 2,304 bytes and its fixed part (barrier, masks, maximum)
// as long as for d 128.
#pragma once

#include "kv4_plan.cuh"
#include "tc_ops.cuh"

namespace sv {

constexpr int KA_WARPS = 4;
constexpr float KA_LIFT = 7.f;                  // log2 of the largest probability when the reference moves
constexpr float KA_TOP = 15.f;                  // and of the largest before it moves

template <int D, int NQ>
struct KaShape {
    static constexpr int ROWS = 8 * NQ;                 // packed rows of an item
    static constexpr int STAGES = D == 64 ? 4 : D == 128 ? 3 : 2;
    // blocks on a multiprocessor, by registers and shared memory
    static constexpr int BLOCKS = D == 64 ? (NQ == 1 ? 5 : 4) : D == 128 ? (NQ == 1 ? 4 : 3) : NQ == 1 ? 3 : 2;
    static constexpr int STAGE = kv_head_bytes(D);
    static constexpr int KSTEPS = D / 16;
    static constexpr int SECTIONS = D == 256 ? 2 : 1;   // of 128 dimensions (64) of the queries and keys
    static constexpr int SK = KSTEPS / SECTIONS;        // K steps of a section
    static constexpr int VN = D / 8;                    // dimensions of a thread's rows
    static constexpr bool STORED = D == 256 && NQ == 2; // the queries are in shared memory
    // shared memory: rings (a warp's sums at an item's end), two warps'
    // statistics, queries, barriers
    static constexpr int RING = STAGES * STAGE;
    static constexpr int STATS = KA_WARPS * RING;
    static constexpr int QUERIES = STATS + 2 * ROWS * 8;
    static constexpr int BARS = QUERIES + (STORED ? KSTEPS * 512 : 0);
    static constexpr int BYTES = BARS + 8 * KA_WARPS * STAGES;
    static_assert(RING >= ROWS * D * 4, "a warp's sums fit its ring");
};

__device__ __forceinline__ float ka_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two probabilities as an fp16 pair.  (Scores past 2^23, whose fp32 steps are
// as wide as the slack, may pass fp16's range: its largest number then.)
__device__ __forceinline__ uint32_t ka_pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The token (of 8) that row n of a half tile of scores stands for.  Those of
// neighbouring rows differ in parity, and four threads' are two even, two odd:
// with 64 bytes a token, no bank conflict among the loads of keys and two ways
// among those of values.
__device__ __forceinline__ int ka_token(int n) { return n & 1 ? 4 + ((n >> 1) ^ 1) : n >> 1; }

// The codes of a token's part that a thread takes: N words, with the widest load.
template <int N>
__device__ __forceinline__ void ka_words(const uint8_t *at, uint32_t (&w)[N])
{
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(at);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(at);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(at);
    }
}

// An 8 x 8 matrix of 16-bit values, a row's neighbours in a register, transposed.
__device__ __forceinline__ uint32_t ka_transpose(uint32_t a)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

template <int D, int NQ>
struct KaWarp {
    using S = KaShape<D, NQ>;
    static constexpr int MT = D / 16;
    float o[MT][NQ][4];                         // dimensions 2 i, 2 i + 1 of the thread's: rows 2c, 2c + 1 of the first, of the second
    float m[NQ][2], l[NQ][2];                   // rows 2c, 2c + 1: reference, KA_LIFT below a maximum; this thread's sum

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int q = 0; q < NQ; ++q) o[i][q][0] = o[i][q][1] = o[i][q][2] = o[i][q][3] = 0.f;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            m[q][0] = m[q][1] = -INFINITY;
            l[q][0] = l[q][1] = 0.f;
        }
    }

    // A page in shared memory: tokens at positions first .. first + 31; row r
    // sees those up to pos[r] that are in its window or among the sinks.
    // `all`: every row sees every token.
    template <class Query>
    __device__ __forceinline__ void page(const uint8_t *st, const Query &query, int first, bool all, const int (&pos)[NQ][2],
                                         const int (&low)[NQ][2], int sinks, const float (&scale)[NQ][2])
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        float s[2][NQ][4];                      // 16 tokens each: rows g and g + 8
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < NQ; ++q) s[j][q][0] = s[j][q][1] = s[j][q][2] = s[j][q][3] = 0.f;
#pragma unroll
        for (int sec = 0; sec < S::SECTIONS; ++sec) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t w[2][S::SK / 2], s2[2][2];     // the scales of the steps' first and second half, twice each
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = 16 * j + 8 * h + ka_token(g);
                    ka_words(st + t * (D / 2) + sec * 64 + c * (2 * S::SK), w[h]);
                    if constexpr (D == 64) {
                        const uint32_t b = st[kv_k_scales(D) + t * 4 + c];
                        s2[h][0] = s2[h][1] = kv_scales2(b | b << 8);
                    } else {
                        const uint32_t v = kv_scales2(*reinterpret_cast<const uint16_t *>(st + kv_k_scales(D) + t * (D / 16) + sec * 8 + 2 * c));
                        s2[h][0] = __byte_perm(v, v, 0x1010);
                        s2[h][1] = __byte_perm(v, v, 0x3232);
                    }
                }
#pragma unroll
                for (int i = 0; i < S::SK / 2; ++i) {
                    uint32_t v[2][4];
                    kv_values8(w[0][i], v[0]);
                    kv_values8(w[1][i], v[1]);
                    const uint32_t f0 = s2[0][2 * i >= S::SK / 2], f1 = s2[1][2 * i >= S::SK / 2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t a0 = kv_mul2(v[0][2 * e], f0), a1 = kv_mul2(v[1][2 * e], f1);
                        const uint32_t a2 = kv_mul2(v[0][2 * e + 1], f0), a3 = kv_mul2(v[1][2 * e + 1], f1);
                        uint32_t b[2 * NQ];
                        query(sec * S::SK + 2 * i + e, b);
#pragma unroll
                        for (int q = 0; q < NQ; ++q) mma_f16_16816(s[j][q], a0, a1, a2, a3, b[2 * q], b[2 * q + 1]);
                    }
                }
            }
        }
        // in units of log2, masked
        float top[NQ][2];
        bool grow = false;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[q][r] = -INFINITY;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = s[j][q][2 * h + r] * scale[q][r];
                        if (!all) {
                            const int t = first + 16 * j + 8 * h + ka_token(g);
                            x = t <= pos[q][r] && (t >= low[q][r] || t < sinks) ? x : -INFINITY;
                        }
                        s[j][q][2 * h + r] = x;
                        top[q][r] = fmaxf(top[q][r], x);
                    }
                // (with -inf before: 0 scores further are enough)
                grow |= top[q][r] > (m[q][r] == -INFINITY ? -INFINITY : m[q][r] + KA_TOP);
            }
        if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float x = top[q][r];
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                    const float to = fmaxf(m[q][r], x - KA_LIFT);
                    f[r] = to == m[q][r] ? 1.f : m[q][r] == -INFINITY ? 0.f : ka_exp2(m[q][r] - to);   // (0: nothing was added before)
                    m[q][r] = to;
                    l[q][r] *= f[r];
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[i][q][0] *= f[0];
                    o[i][q][1] *= f[1];
                    o[i][q][2] *= f[0];
                    o[i][q][3] *= f[1];
                }
            }
        }
        uint32_t p[2][NQ][2];                   // 16 tokens: tokens 2c, 2c + 1 of row g, 2c + 8, 2c + 9
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const float ref[2] = {m[q][0] == -INFINITY ? 0.f : m[q][0], m[q][1] == -INFINITY ? 0.f : m[q][1]};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = ka_exp2(s[j][q][2 * h] - ref[0]), y = ka_exp2(s[j][q][2 * h + 1] - ref[1]);
                    l[q][0] += x;
                    l[q][1] += y;
                    p[j][q][h] = ka_transpose(ka_pack(x, y));
                }
        }
        const uint8_t *vc = st + kv_v_codes(D) + g * (S::VN / 2), *vs = st + kv_v_scales(D) + g * S::VN / KV_GROUP;
#pragma unroll
        for (int k = 0; k < 2; ++k) {           // 16 tokens
            constexpr int W = S::VN / 8, GROUPS = S::VN > 16 ? S::VN / 16 : 1;
            uint32_t w[4][W], f[GROUPS][2];
            uint32_t sc[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {       // tokens 2c, 2c + 1, 2c + 8, 2c + 9
                const int t = 16 * k + 8 * (q >> 1) + ka_token(2 * c + (q & 1));
                ka_words(vc + t * (D / 2), w[q]);
                sc[q] = GROUPS == 2 ? *reinterpret_cast<const uint16_t *>(vs + t * (D / 16)) : vs[t * (D / 16)];
            }
#pragma unroll
            for (int n = 0; n < GROUPS; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    f[n][q] = kv_finite2(kv_scales2(__byte_perm(sc[2 * q], sc[2 * q + 1], n ? 0x0051 : 0x0040)));
#pragma unroll
            for (int i = 0; i < W; ++i) {
                uint32_t v[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) kv_values8(w[q][i], v[q]);
                const int n = GROUPS == 2 ? i / 2 : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a0 = kv_mul2(__byte_perm(v[0][j], v[1][j], 0x5410), f[n][0]);
                    const uint32_t a1 = kv_mul2(__byte_perm(v[0][j], v[1][j], 0x7632), f[n][0]);
                    const uint32_t a2 = kv_mul2(__byte_perm(v[2][j], v[3][j], 0x5410), f[n][1]);
                    const uint32_t a3 = kv_mul2(__byte_perm(v[2][j], v[3][j], 0x7632), f[n][1]);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) mma_f16_16816(o[4 * i + j][q], a0, a1, a2, a3, p[k][q][0], p[k][q][1]);
                }
            }
        }
    }
};

template <int D, int NQ>
__global__ void __launch_bounds__(KA_WARPS * 32, (KaShape<D, NQ>::BLOCKS)) kv4_attn_kernel(const KvAttnParams p)
{
    using S = KaShape<D, NQ>;
    extern __shared__ __align__(128) uint8_t ka_smem[];
    __shared__ volatile int failed;
    const TcWait wait{&failed, p.err};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t *ring = ka_smem + warp * S::RING;
    const uint32_t bars = smem_addr(ka_smem + S::BARS) + 8 * warp * S::STAGES;
    if (threadIdx.x == 0) {
        failed = 0;
        for (int i = 0; i < KA_WARPS * S::STAGES; ++i) mbar_init(smem_addr(ka_smem + S::BARS) + 8 * i, 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait_prior();
    const uint64_t policy = policy_evict_first();
    // (found in what the rings are later)
    static_assert(sizeof(KvPartSmem) <= S::STATS, "room for the parts");
    KvPart part = kv_part(p, *reinterpret_cast<KvPartSmem *>(ka_smem));
    fence_proxy_async();
    __syncthreads();
    if (threadIdx.x == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    uint32_t phases = 0;                        // bit i: the parity that stage i completes next

    while (part.left > 0) {
        const KvItem &it = part.item;
        const int u0 = part.unit, n = part.n;
        const int mine = n > warp ? (n - warp + KA_WARPS - 1) / KA_WARPS : 0;   // this warp's pages
        // its i-th page's place in the sequence, and its entry in the table
        auto place = [&](int i) { return it.span.at(u0 + warp + KA_WARPS * i); };
        const int32_t *table = p.kv.table + it.b * p.kv.ldt;
        const int pages = it.seq.before < 0 ? 0 : p.kv.max_pages;
        auto entry = [&](int i) { return i < mine && place(i) < pages ? table[place(i)] : -1; };
        const uint8_t *head = p.kv.pages + static_cast<long long>(it.h) * S::STAGE;
        const long long stride = static_cast<long long>(p.kv.Hk) * S::STAGE;
        uint32_t there = 0;                     // bit i: stage i holds a page
        int at_in = 0, at = 0;                  // stages: of the next copy, of the next page
        auto ask = [&](int id) {
            if (id >= 0 && id < p.kv.n_pages) {
                there |= 1u << at_in;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bars + 8 * at_in, S::STAGE);
                    bulk_g2s(smem_addr(ring) + at_in * S::STAGE, head + id * stride, S::STAGE, bars + 8 * at_in, policy);
                }
            } else {
                there &= ~(1u << at_in);
                if (it.seq.before >= 0 && lane == 0) atomicOr(p.err, KV_ERR_PAGE);
            }
            if (++at_in == S::STAGES) at_in = 0;
        };
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i)
            if (i < mine) ask(entry(i));
        int id_next = entry(S::STAGES - 1);     // (read a page ahead)

        // the tile's queries: this thread has row g of each eight
        const int rows = min(S::ROWS, it.seq.n * p.G - it.tile * S::ROWS);
        uint32_t b[S::STORED ? 1 : S::KSTEPS][2 * NQ];
        float scale_g[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int row = 8 * q + g, packed = it.tile * S::ROWS + row, t = kv_token(p, packed), hq = packed - t * p.G;
            const bool in = row < rows;
            const uint4 *at = reinterpret_cast<const uint4 *>(p.q + (it.seq.first + (in ? t : 0)) * p.ldq +
                                                              static_cast<long long>(it.h * p.G + (in ? hq : 0)) * D);
            unsigned top = 0;
#pragma unroll
            for (int sec = 0; sec < S::SECTIONS; ++sec)
#pragma unroll
                for (int i = 0; i < S::SK / 2; ++i) {
                    const uint4 v = in ? at[sec * 16 + c * (S::SK / 2) + i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
                }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int shift = xres_shift(top);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
            scale_g[q] = p.scale * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
            for (int sec = 0; sec < S::SECTIONS; ++sec)
#pragma unroll
                for (int i = 0; i < S::SK / 2; ++i) {
                    const uint4 v = in ? at[sec * 16 + c * (S::SK / 2) + i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = pack_f16x2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
                        const int k = sec * S::SK + 2 * i + (e >> 1), reg = 2 * q + (e & 1);
                        if constexpr (!S::STORED)
                            b[k][reg] = x;
                        else if (warp == 0)
                            reinterpret_cast<uint32_t *>(ka_smem + S::QUERIES)[(k * 32 + lane) * 4 + reg] = x;
                    }
                }
        }
        if constexpr (S::STORED) __syncthreads();
        auto query = [&](int k, uint32_t (&to)[2 * NQ]) {
            if constexpr (!S::STORED) {
#pragma unroll
                for (int e = 0; e < 2 * NQ; ++e) to[e] = b[k][e];
            } else {
                const uint4 v = reinterpret_cast<const uint4 *>(ka_smem + S::QUERIES)[k * 32 + lane];
                to[0] = v.x, to[1] = v.y, to[2 * NQ - 2] = v.z, to[2 * NQ - 1] = v.w;
            }
        };
        // the softmax's rows: 2c and 2c + 1 of each eight
        int pos[NQ][2], low[NQ][2];
        float scale[NQ][2];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 8 * q + 2 * c + r;
                pos[q][r] = row < rows && it.seq.before >= 0 ? it.seq.before + kv_token(p, it.tile * S::ROWS + row) : -1;
                low[q][r] = p.window > 0 ? pos[q][r] - p.window + 1 : 0;
                scale[q][r] = __shfl_sync(0xFFFFFFFFu, scale_g[q], 4 * (2 * c + r));
            }
        // tokens that every row of the tile sees: from .. to, and below the sinks
        const int t0 = kv_token(p, it.tile * S::ROWS), t1 = kv_token(p, it.tile * S::ROWS + rows - 1);
        const int to = it.seq.before < 0 ? -1 : it.seq.before + t0;
        const int from = p.window > 0 ? it.seq.before + t1 - p.window + 1 : 0;

        if (threadIdx.x == 0 && it.seq.before >= 0 && it.seq.before + t1 >= p.kv.max_pages * KV_PAGE) atomicOr(p.err, KV_ERR_PAGE);
        const int sinks = p.window > 0 ? p.sinks : 0;
        KaWarp<D, NQ> w;
        w.clear();
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            fence_proxy_async();                // (the stage has been read before a copy may write there)
            __syncwarp();
            if (i + S::STAGES - 1 < mine) {
                ask(id_next);
                id_next = entry(i + S::STAGES);
            }
            if (there >> at & 1) {
                wait(bars + 8 * at, phases >> at);
                phases ^= 1u << at;
                const int first = KV_PAGE * place(i);
                const bool all = first + KV_PAGE - 1 <= to && (first >= from || first + KV_PAGE <= p.sinks);
                w.page(ring + at * S::STAGE, query, first, all, pos, low, sinks, scale);
            }
            if (++at == S::STAGES) at = 0;
        }
        __syncwarp();

        // the warps' sums: 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) w.l[q][r] += __shfl_xor_sync(0xFFFFFFFFu, w.l[q][r], x);
        float2 *stats = reinterpret_cast<float2 *>(ka_smem + S::STATS);
        for (int half = KA_WARPS / 2; half; half >>= 1) {
            if (warp >= half && warp < 2 * half) {
                const int at = (warp - half) * S::ROWS;
                if (g == 0) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int r = 0; r < 2; ++r) stats[at + 8 * q + 2 * c + r] = make_float2(w.m[q][r], w.l[q][r]);
                }
                float4 *sums = reinterpret_cast<float4 *>(ring);
#pragma unroll
                for (int i = 0; i < w.MT; ++i)
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
                        sums[(i * NQ + q) * 32 + lane] = make_float4(w.o[i][q][0], w.o[i][q][1], w.o[i][q][2], w.o[i][q][3]);
                fence_proxy_async();            // (the ring's next copies come after)
            }
            __syncthreads();
            if (warp < half) {
                const float4 *sums = reinterpret_cast<const float4 *>(ring + half * S::RING);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    float f[2], e[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 x = stats[warp * S::ROWS + 8 * q + 2 * c + r];
                        const float top = fmaxf(w.m[q][r], x.x), ref = top == -INFINITY ? 0.f : top;
                        f[r] = ka_exp2(w.m[q][r] - ref);
                        e[r] = ka_exp2(x.x - ref);
                        w.m[q][r] = top;
                        w.l[q][r] = f[r] * w.l[q][r] + e[r] * x.y;
                    }
#pragma unroll
                    for (int i = 0; i < w.MT; ++i) {
                        const float4 v = sums[(i * NQ + q) * 32 + lane];
                        w.o[i][q][0] = f[0] * w.o[i][q][0] + e[0] * v.x;
                        w.o[i][q][1] = f[1] * w.o[i][q][1] + e[1] * v.y;
                        w.o[i][q][2] = f[0] * w.o[i][q][2] + e[0] * v.z;
                        w.o[i][q][3] = f[1] * w.o[i][q][3] + e[1] * v.w;
                    }
                }
                fence_proxy_async();
            }
            __syncthreads();
        }
        if (warp == 0) {
            const bool whole = part.whole();
            const int slot = 2 * blockIdx.x + (part.unit == 0);
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = 8 * q + 2 * c + r, packed = it.tile * S::ROWS + row, t = kv_token(p, packed), hq = packed - t * p.G;
                    if (row >= rows) continue;
                    if (whole) {
                        const float f = w.l[q][r] == 0.f ? 0.f : p.v_scale / w.l[q][r];
                        uint4 *o = reinterpret_cast<uint4 *>(p.o + (it.seq.first + t) * p.ldo +
                                                             static_cast<long long>(it.h * p.G + hq) * D + g * S::VN);
#pragma unroll
                        for (int i = 0; i < S::VN / 8; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[e])
                                    : "f"(w.o[4 * i + e][q][2 + r] * f), "f"(w.o[4 * i + e][q][r] * f));
                            o[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
                        float4 *o = reinterpret_cast<float4 *>(p.sums + (static_cast<long long>(slot) * S::ROWS + row) * D + g * S::VN);
#pragma unroll
                        for (int i = 0; i < S::VN / 4; ++i)
                            o[i] = make_float4(w.o[2 * i][q][r], w.o[2 * i][q][2 + r], w.o[2 * i + 1][q][r], w.o[2 * i + 1][q][2 + r]);
                        if (g == 0)
                            reinterpret_cast<float2 *>(p.stats)[static_cast<long long>(slot) * S::ROWS + row] = make_float2(w.m[q][r], w.l[q][r]);
                    }
                }
            if (lane == 0 && part.parts() > 1) p.joins[blockIdx.x] = make_int4(part.parts(), it.h, it.b, it.tile);
        }
        part.next(p);
    }
    // (only now: a join's blocks would wait in the places of later blocks of this kernel)
    pdl_launch_dependents();
}

}  // namespace sv
