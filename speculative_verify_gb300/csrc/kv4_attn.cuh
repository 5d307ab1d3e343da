// kv4_attn.cuh -- attention of a few query rows over the 4-bit cache, straight
// from the packed pages on mma.sync: o = softmax(scale q k^T) v, row by row
// over the tokens that it sees.
//
// A warp takes a page of its head's item (kv4_plan.cuh) at a time, from a ring
// of its own filled by bulk copies, and keeps a running softmax of its own; the
// warps of a block join at the item's end.  Products are m16n8k16 of fp16: rows
// are up to 16 packed query rows.  Keys and values become fp16 in registers,
// exactly (kv4.cuh): one conversion and one product a pair.
//   * Scores: a thread's B column is a token and its K steps are that token's
//     32 neighbouring dimensions, so a token's codes come in one 16-byte load.
//     Queries are laid out the same, times a power of two of their row that
//     puts the largest in [2^14, 2^15): exact but for values 2^-25 of it.
//   * Values: probabilities are the A operand as the score product leaves
//     them, and a B column is a dimension; a pair of tokens' values are put
//     together by byte permutation.  Thread column n has dimensions n d / 8 ..,
//     so that it ends with neighbouring ones.
//   * Sums and the softmax are fp32, probabilities fp16 (2^-12 of each,
//     independent).  They are taken relative to a maximum that is only moved
//     when a score passes it by 2^8, so most pages rescale nothing.
#pragma once

#include "kv4_plan.cuh"
#include "tc_ops.cuh"

namespace sv {

constexpr int KA_WARPS = 4;
constexpr int KA_ROWS = 16;                     // packed rows of an item
constexpr float KA_SLACK = 8.f;                 // log2 of the largest probability

template <int D>
struct KaShape {
    static constexpr int STAGES = D == 64 ? 4 : D == 128 ? 3 : 2;
    static constexpr int BLOCKS = D == 64 ? 4 : D == 128 ? 3 : 2;   // on a multiprocessor
    static constexpr int STAGE = kv_head_bytes(D);
    static constexpr int KSTEPS = D / 16;
    static constexpr int SECTIONS = D == 256 ? 2 : 1;   // of 128 dimensions (64) of the queries and keys
    static constexpr int SK = KSTEPS / SECTIONS;        // K steps of a section
    static constexpr int VN = D / 8;                    // dimensions of a thread's value column
    // shared memory: rings (a warp's sums at an item's end), two warps'
    // statistics, queries (SECTIONS > 1), barriers
    static constexpr int RING = STAGES * STAGE;
    static constexpr int STATS = KA_WARPS * RING;
    static constexpr int QUERIES = STATS + 2 * KA_ROWS * 8;
    static constexpr int BARS = QUERIES + (SECTIONS > 1 ? KSTEPS * 512 : 0);
    static constexpr int BYTES = BARS + 8 * KA_WARPS * STAGES;
    static_assert(RING >= KA_ROWS * D * 4, "a warp's sums fit its ring");
};

__device__ __forceinline__ float ka_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The token (of 8) that column n of a score tile stands for.  Rows of
// neighbouring columns differ in parity, and four threads' rows are two even,
// two odd: with 64 bytes a token, no bank conflict among the loads of keys and
// two ways among those of values.
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

template <int D>
struct KaWarp {
    using S = KaShape<D>;
    float o[S::VN][4];                          // dimension n VN + i: rows g, columns 2c, 2c + 1; rows g + 8
    float m[2], l[2];                           // reference maximum, this thread's sum; rows g, g + 8

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < S::VN; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // A page in shared memory: tokens at positions first .. first + 31; row r
    // sees those up to pos[r] that are in its window or among the sinks.
    // `all`: every row sees every token.
    template <class Query>
    __device__ __forceinline__ void page(const uint8_t *st, const Query &query, int first, bool all, const int (&pos)[2],
                                         const int (&low)[2], int sinks, const float (&scale)[2])
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int sec = 0; sec < S::SECTIONS; ++sec) {
            uint32_t a[S::SK][4];
            query(sec, a);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 8 * j + ka_token(g);
                uint32_t w[S::SK / 2];
                ka_words(st + t * (D / 2) + sec * 64 + c * (2 * S::SK), w);
                uint32_t s2[2];                 // the scales of the steps' first and second half, twice each
                if constexpr (D == 64) {
                    const uint32_t b = st[kv_k_scales(D) + t * 4 + c];
                    s2[0] = s2[1] = kv_scales2(b | b << 8);
                } else {
                    const uint32_t v = kv_scales2(*reinterpret_cast<const uint16_t *>(st + kv_k_scales(D) + t * (D / 16) + sec * 8 + 2 * c));
                    s2[0] = __byte_perm(v, v, 0x1010);
                    s2[1] = __byte_perm(v, v, 0x3232);
                }
#pragma unroll
                for (int i = 0; i < S::SK / 2; ++i) {
                    uint32_t v[4];
                    kv_values8(w[i], v);
                    const uint32_t f = s2[2 * i >= S::SK / 2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        mma_f16_16816(s[j], a[2 * i + e][0], a[2 * i + e][1], a[2 * i + e][2], a[2 * i + e][3],
                                      kv_mul2(v[2 * e], f), kv_mul2(v[2 * e + 1], f));
                }
            }
        }
        // in units of log2, masked
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = e >> 1;
                float x = s[j][e] * scale[r];
                if (!all) {
                    const int t = first + 8 * j + ka_token(2 * c + (e & 1));
                    x = t <= pos[r] && (t >= low[r] || t < sinks) ? x : -INFINITY;
                }
                s[j][e] = x;
                top[r] = fmaxf(top[r], x);
            }
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + KA_SLACK || top[1] > m[1] + KA_SLACK || (top[0] > m[0] && m[0] == -INFINITY) ||
                                        (top[1] > m[1] && m[1] == -INFINITY))) {
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
                const float to = fmaxf(m[r], top[r]);
                f[r] = m[r] == -INFINITY ? 0.f : ka_exp2(m[r] - to);    // (nothing was added before)
                f[r] = to == m[r] ? 1.f : f[r];
                m[r] = to;
                l[r] *= f[r];
            }
#pragma unroll
            for (int i = 0; i < S::VN; ++i) {
                o[i][0] *= f[0];
                o[i][1] *= f[0];
                o[i][2] *= f[1];
                o[i][3] *= f[1];
            }
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        uint32_t p[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float x = ka_exp2(s[j][2 * r] - ref[r]), y = ka_exp2(s[j][2 * r + 1] - ref[r]);
                l[r] += x + y;
                p[j][r] = pack_f16x2(x, y);
            }
        const uint8_t *vc = st + kv_v_codes(D) + g * (S::VN / 2), *vs = st + kv_v_scales(D) + g * S::VN / KV_GROUP;
#pragma unroll
        for (int k = 0; k < 2; ++k) {           // 16 tokens
            constexpr int W = S::VN / 8, GROUPS = S::VN > 16 ? S::VN / 16 : 1;
            uint32_t w[4][W], f[GROUPS][2];
            uint32_t sc[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {       // tile 2k's columns 2c, 2c + 1, tile 2k + 1's
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
                    const uint32_t b0 = kv_mul2(__byte_perm(v[0][j], v[1][j], 0x5410), f[n][0]);
                    const uint32_t b1 = kv_mul2(__byte_perm(v[2][j], v[3][j], 0x5410), f[n][1]);
                    mma_f16_16816(o[8 * i + 2 * j], p[2 * k][0], p[2 * k][1], p[2 * k + 1][0], p[2 * k + 1][1], b0, b1);
                    const uint32_t c0 = kv_mul2(__byte_perm(v[0][j], v[1][j], 0x7632), f[n][0]);
                    const uint32_t c1 = kv_mul2(__byte_perm(v[2][j], v[3][j], 0x7632), f[n][1]);
                    mma_f16_16816(o[8 * i + 2 * j + 1], p[2 * k][0], p[2 * k][1], p[2 * k + 1][0], p[2 * k + 1][1], c0, c1);
                }
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(KA_WARPS * 32, KaShape<D>::BLOCKS) kv4_attn_kernel(const KvAttnParams p)
{
    using S = KaShape<D>;
    extern __shared__ __align__(128) uint8_t ka_smem[];
    __shared__ volatile int failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t *ring = ka_smem + warp * S::RING;
    const uint32_t bars = smem_addr(ka_smem + S::BARS) + 8 * warp * S::STAGES;
    if (threadIdx.x == 0) {
        failed = 0;
        for (int i = 0; i < KA_WARPS * S::STAGES; ++i) mbar_init(smem_addr(ka_smem + S::BARS) + 8 * i, 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_prior();
    const uint64_t policy = policy_evict_first();
    __shared__ KvPartSmem part_sm;
    KvPart part = kv_part(p, part_sm);
    if (threadIdx.x == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    uint32_t phases = 0;                        // bit i: the parity that stage i completes next

    while (part.left > 0) {
        const KvItem &it = part.item;
        const int u0 = it.unit, n = part.units();
        const int mine = n > warp ? (n - warp + KA_WARPS - 1) / KA_WARPS : 0;   // this warp's pages
        auto page_of = [&](int i) { return it.seq.before < 0 ? -1 : p.kv.at(it.b, it.span.at(u0 + warp + KA_WARPS * i)); };
        uint32_t there = 0;
        auto ask = [&](int i, int page) {
            const int st = i % S::STAGES;
            if (page < 0) {
                there &= ~(1u << st);
                if (it.seq.before >= 0 && lane == 0) atomicOr(p.err, KV_ERR_PAGE);
                return;
            }
            there |= 1u << st;
            if (lane == 0) {
                mbar_arrive_expect_tx(bars + 8 * st, S::STAGE);
                bulk_g2s(smem_addr(ring + st * S::STAGE), p.kv.head<D>(page, it.h), S::STAGE, bars + 8 * st, policy);
            }
        };
        for (int i = 0; i < S::STAGES - 1 && i < mine; ++i) ask(i, page_of(i));

        // the tile's rows: this thread has rows g and g + 8
        const int rows = min(KA_ROWS, it.seq.n * p.G - it.tile * KA_ROWS);
        int pos[2], low[2];
        float scale[2];
        uint32_t a[S::SK][4];                   // (one section: kept)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r, packed = it.tile * KA_ROWS + row, t = kv_token(p, packed), hq = packed - t * p.G;
            const bool in = row < rows;
            pos[r] = in && it.seq.before >= 0 ? it.seq.before + t : -1;
            low[r] = p.window > 0 ? pos[r] - p.window + 1 : 0;
            const uint4 *q = reinterpret_cast<const uint4 *>(p.q + (it.seq.first + (in ? t : 0)) * p.ldq +
                                                             static_cast<long long>(it.h * p.G + (in ? hq : 0)) * D);
            unsigned top = 0;
#pragma unroll
            for (int sec = 0; sec < S::SECTIONS; ++sec)
#pragma unroll
                for (int i = 0; i < S::SK / 2; ++i) {
                    const uint4 v = in ? q[sec * 16 + c * (S::SK / 2) + i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
                }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int shift = xres_shift(top);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
            scale[r] = p.scale * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
            for (int sec = 0; sec < S::SECTIONS; ++sec)
#pragma unroll
                for (int i = 0; i < S::SK / 2; ++i) {
                    const uint4 v = in ? q[sec * 16 + c * (S::SK / 2) + i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = pack_f16x2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
                        const int k = 2 * i + (e >> 1), reg = r + 2 * (e & 1);
                        if constexpr (S::SECTIONS == 1)
                            a[k][reg] = x;
                        else if (warp == 0)
                            reinterpret_cast<uint32_t *>(ka_smem + S::QUERIES)[((sec * S::SK + k) * 32 + lane) * 4 + reg] = x;
                    }
                }
        }
        if constexpr (S::SECTIONS > 1) __syncthreads();
        auto query = [&](int sec, uint32_t (&to)[S::SK][4]) {
#pragma unroll
            for (int k = 0; k < S::SK; ++k) {
                if constexpr (S::SECTIONS == 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[k][e] = a[k][e];
                } else {
                    const uint4 v = reinterpret_cast<const uint4 *>(ka_smem + S::QUERIES)[(sec * S::SK + k) * 32 + lane];
                    to[k][0] = v.x, to[k][1] = v.y, to[k][2] = v.z, to[k][3] = v.w;
                }
            }
        };
        // tokens that every row of the tile sees: from .. to, and below `sunk`
        const int t0 = kv_token(p, it.tile * KA_ROWS), t1 = kv_token(p, it.tile * KA_ROWS + rows - 1);
        const int to = it.seq.before < 0 ? -1 : it.seq.before + t0;
        const int from = p.window > 0 ? it.seq.before + t1 - p.window + 1 : 0;

        if (threadIdx.x == 0 && it.seq.before >= 0 && it.seq.before + t1 >= p.kv.max_pages * KV_PAGE) atomicOr(p.err, KV_ERR_PAGE);
        KaWarp<D> w;
        w.clear();
        for (int i = 0; i < mine; ++i) {
            const int nx = i + S::STAGES - 1;
            fence_proxy_async();                // (the stage has been read before a copy may write there)
            __syncwarp();
            if (nx < mine) ask(nx, page_of(nx));
            const int st = i % S::STAGES;
            if (there >> st & 1) {
                if (!mbar_wait_bounded(bars + 8 * st, phases >> st & 1, failed ? WAIT_LIMIT_AFTER_ERR_NS : WAIT_LIMIT_NS)) {
                    failed = 1;
                    atomicOr(p.err, 2);
                }
                phases ^= 1u << st;
                const int first = KV_PAGE * it.span.at(u0 + warp + KA_WARPS * i);
                const bool all = first + KV_PAGE - 1 <= to && (first >= from || first + KV_PAGE <= p.sinks);
                w.page(ring + st * S::STAGE, query, first, all, pos, low, p.window > 0 ? p.sinks : 0, scale);
            }
        }
        __syncwarp();

        // the warps' sums: 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            w.l[r] += __shfl_xor_sync(0xFFFFFFFFu, w.l[r], 1);
            w.l[r] += __shfl_xor_sync(0xFFFFFFFFu, w.l[r], 2);
        }
        float2 *stats = reinterpret_cast<float2 *>(ka_smem + S::STATS);
        for (int half = KA_WARPS / 2; half; half >>= 1) {
            if (warp >= half && warp < 2 * half) {
                const int at = warp - half;
                if (c == 0) {
                    stats[at * KA_ROWS + g] = make_float2(w.m[0], w.l[0]);
                    stats[at * KA_ROWS + g + 8] = make_float2(w.m[1], w.l[1]);
                }
                float4 *sums = reinterpret_cast<float4 *>(ring);
#pragma unroll
                for (int i = 0; i < S::VN; ++i) sums[i * 32 + lane] = make_float4(w.o[i][0], w.o[i][1], w.o[i][2], w.o[i][3]);
                fence_proxy_async();            // (the ring's next copies come after)
            }
            __syncthreads();
            if (warp < half) {
                const float4 *sums = reinterpret_cast<const float4 *>(ring + half * S::RING);
                float f[2], e[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 s = stats[warp * KA_ROWS + g + 8 * r];
                    const float top = fmaxf(w.m[r], s.x), ref = top == -INFINITY ? 0.f : top;
                    f[r] = ka_exp2(w.m[r] - ref);
                    e[r] = ka_exp2(s.x - ref);
                    w.m[r] = top;
                    w.l[r] = f[r] * w.l[r] + e[r] * s.y;
                }
#pragma unroll
                for (int i = 0; i < S::VN; ++i) {
                    const float4 v = sums[i * 32 + lane];
                    w.o[i][0] = f[0] * w.o[i][0] + e[0] * v.x;
                    w.o[i][1] = f[0] * w.o[i][1] + e[0] * v.y;
                    w.o[i][2] = f[1] * w.o[i][2] + e[1] * v.z;
                    w.o[i][3] = f[1] * w.o[i][3] + e[1] * v.w;
                }
            }
            __syncthreads();
        }
        if (warp == 0) {
            const bool whole = part.whole();
            const int slot = 2 * blockIdx.x + (it.unit == 0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r, packed = it.tile * KA_ROWS + row, t = kv_token(p, packed), hq = packed - t * p.G;
                if (row >= rows) continue;
                if (whole) {
                    const float f = w.l[r] == 0.f ? 0.f : p.v_scale / w.l[r];
                    // columns 2c and 2c + 1: 2 VN neighbouring dimensions
                    uint4 *o = reinterpret_cast<uint4 *>(p.o + (it.seq.first + t) * p.ldo +
                                                         static_cast<long long>(it.h * p.G + hq) * D + 2 * c * S::VN);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < S::VN / 8; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[e])
                                    : "f"(w.o[8 * i + 2 * e + 1][2 * r + k] * f), "f"(w.o[8 * i + 2 * e][2 * r + k] * f));
                            o[k * (S::VN / 8) + i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                } else {
                    float4 *o = reinterpret_cast<float4 *>(p.sums + (static_cast<long long>(slot) * KA_ROWS + row) * D + 2 * c * S::VN);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < S::VN / 4; ++i)
                            o[k * (S::VN / 4) + i] = make_float4(w.o[4 * i][2 * r + k], w.o[4 * i + 1][2 * r + k],
                                                                 w.o[4 * i + 2][2 * r + k], w.o[4 * i + 3][2 * r + k]);
                    if (c == 0)
                        reinterpret_cast<float2 *>(p.stats)[static_cast<long long>(slot) * KA_ROWS + row] = make_float2(w.m[r], w.l[r]);
                }
            }
            if (lane == 0 && part.parts() > 1) p.joins[blockIdx.x] = make_int4(part.parts(), it.h, it.b, it.tile);
        }
        part.next(p);
    }
}

}  // namespace sv
