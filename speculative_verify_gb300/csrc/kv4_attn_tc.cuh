// kv4_attn_tc.cuh -- attention of many query rows over the 4-bit cache on the
// 5th-generation tensor cores: prompts, and verify rows with many packed rows
// (attn_plan in attn_ops.cu has the rule).
//
// An item (kv4_plan.cuh) is NT tiles of 128 packed rows, a unit 64 tokens.  A
// unit's keys and its values become fp16 in shared memory once for all tiles,
// exactly (kv4.cuh), as blocks of a ring in the order in which the products use
// them.  Scores S = Q K^T (M128 N64) go to tensor memory, one buffer while the
// softmax warps turn the other's into fp16 probabilities, in the same columns;
// O += P V takes P from tensor memory and V across.  So the tensor cores form
// the next unit's scores during a softmax.
//
// NT = 2 (d 64 and 128, many rows): O and two buffers of S for each
// tile fill the tensor memory, and the queries stay in shared memory.  NT = 1
// (fewer rows, or d 256): the queries are in tensor memory too -- from shared
// memory they would take as much of its bandwidth as an M128 N64 product has.
//
// The softmax is that of kv4_attn.cuh: fp32, relative to 2^-7 of a maximum that
// moves only when a score passes it by 2^8, when O is rescaled in tensor memory
// by the rows' own threads.
//
// Roles: the first 8 warps queries, softmax, O and outputs (a thread a row with
// two tiles, two with one); then codes to fp16; products; copies (bulk copies
// of the pages' codes and scales).
//
// d 256 is bound by shared memory: a unit's keys and values are 64 KB of fp16,
// written once and read once by the products, and with the codes they take 70 %
// of its cycles; d 128 with two tiles by the hand-offs between softmax and
// products.  8,192 rows of 24 query heads (4 of 256) from nothing take 743 us,
// 1.1 PFLOP/s; 2,048 rows of 32 (8 of 128) in a window of 4,096 179 us, 0.78;
// nine ragged prompts after 500 tokens each (4,817 rows, same heads) 161 us.
// Verify rows, of which a tile has few: 1 x 4 rows of 131,072 tokens (24 heads
// over 4 of 256) 80 us, 4 x 8 rows of 16,384 45 us.  No pipe is full there
// (shared memory 54 % of its cycles, tensor cores 42): the softmax goes through
// all 128 rows of a tile and its warps meet once a unit.
#pragma once

#include "kv4_attn.cuh"
#include "kv4_plan.cuh"
#include "tc_ops.cuh"

namespace sv {

constexpr int KT_ROWS = 128;                    // packed rows of a tile
constexpr int KT_UNIT = 64;                     // tokens of a unit, and of a ring block

// Warps.  18 with one tile, 96 registers a thread; 14 with two, 128.
template <int NT>
struct KtWarps {
    static constexpr int SOFT = 8, CODE = NT == 2 ? 4 : 8;
    static constexpr int MMA = SOFT + CODE, COPY = MMA + 1, THREADS = 32 * (COPY + 1);
    static constexpr int TILE = SOFT / NT;      // softmax warps of a tile
};

template <int D, int NT>
struct KtSmem {
    static constexpr int BLOCK = KT_UNIT * D * 2;       // fp16 of a unit's keys or values
    static constexpr int BLOCKS = D == 256 ? 4 : 8;
    // codes and scales of an entry's tokens; each conversion group has a ring of
    // its own
    static constexpr int PIECES = D == 256 ? 2 : 1;     // entries of a block
    static constexpr int ENTRY = KT_UNIT / PIECES * (D / 2 + D / 16);
    static constexpr int TURN = 3, ENTRIES = 2 * TURN;  // entries of a group, and of both
    static constexpr int Q = NT * KT_ROWS * D * 2;
    static constexpr int RING = Q, RAW = RING + BLOCKS * BLOCK, STAT = RAW + ENTRIES * ENTRY;
    static constexpr int FACTOR = STAT + 6 * KT_ROWS * 4;       // scores' factors of the rows
    static constexpr int MASK = FACTOR + NT * KT_ROWS * 4;          // missing pages of the last 16 units
    static constexpr int BARS = MASK + 16 * 2;
    // barriers
    static constexpr int RAW_FULL = 0, RAW_EMPTY = ENTRIES, B_FULL = 2 * ENTRIES, B_EMPTY = B_FULL + BLOCKS,
                         S_FULL = B_EMPTY + BLOCKS, P_FULL = S_FULL + 2 * NT, O_DONE = P_FULL + 2 * NT,
                         Q_FULL = O_DONE + 2 * NT, COUNT = Q_FULL + NT;
    static constexpr int USED = BARS + 8 * COUNT + 16;
    // (more than half of a multiprocessor's: two blocks would wait for each other's tensor memory)
    static constexpr int BYTES = USED > 116 * 1024 ? USED : 116 * 1024;
    static_assert(BYTES <= 232448, "shared memory of a block");
    // tensor memory: O of the tiles, the queries (one tile), two S a tile
    static constexpr uint32_t O(int tile) { return static_cast<uint32_t>(tile * D); }
    static constexpr uint32_t QUERY = NT * D;
    static constexpr uint32_t S(int tile, int i) { return static_cast<uint32_t>(NT * D + (NT == 1 ? D / 2 : 0) + 64 * (2 * tile + i)); }
    static constexpr int TMEM = 512;
    static_assert(S(NT - 1, 1) + 64 <= TMEM, "tensor memory");
};

// Instruction descriptor of an M = 128 product of n columns, fp16 operands.
constexpr uint32_t kt_idesc(int n, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Descriptor of 128-byte swizzled rows (tc_ops.cuh), strides in bytes.
__device__ __forceinline__ uint64_t kt_desc(uint32_t saddr, uint32_t leading, uint32_t stride)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(leading >> 4) << 16) |
           (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// D[tmem] (+)= A[smem] x B[smem], four K steps of 16 (64 columns) 32 bytes
// apart in both; whole-warp form, one elected lane issues.
__device__ __forceinline__ void kt_mma4_ss_warp(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, e, t;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, %10, %10;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, t;\n\t}"
                 ::"r"(d_tmem), "l"(a), "l"(a + 2u), "l"(a + 4u), "l"(a + 6u), "l"(b), "l"(b + 2u), "l"(b + 4u), "l"(b + 6u),
                   "r"(idesc), "r"(accumulate)
                 : "memory");
}

// D[tmem] (+)= A[tmem] x B[smem], four K steps of 16: A 8 columns apart, the
// last two `skip` further, B `step` (in 16 bytes) apart.
__device__ __forceinline__ void kt_mma4_ts_warp(uint32_t d_tmem, uint32_t a, uint32_t skip, uint64_t b, uint64_t step, uint32_t idesc,
                                                uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, e, t;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, %10, %10;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, t;\n\t}"
                 ::"r"(d_tmem), "r"(a), "r"(a + 8u), "r"(a + 16u + skip), "r"(a + 24u + skip), "l"(b), "l"(b + step), "l"(b + 2u * step),
                   "l"(b + 3u * step), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ f32x2 kt_add_x2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// A ring's place, and how many times the ring has been round.
template <int N>
struct KtTurn {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == N) {
            at = 0;
            ++round;
        }
    }
};

// What a row sees: tokens up to pos in its window, from `low` on, or below `sinks`.
struct KtSight {
    int pos, low, sinks;
    // The bits below n of 32.
    static __device__ __forceinline__ unsigned below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }
    // Bit i: token first + i is seen.  (first is a page's first; bit 0 of `missing`: the page is not there)
    __device__ __forceinline__ unsigned operator()(int first, unsigned missing) const
    {
        const unsigned seen = below(pos - first + 1) & (~below(low - first) | below(sinks - first));
        return missing & 1u ? 0u : seen;
    }
};

// Scores times a factor, those that are not seen to -inf.
__device__ __forceinline__ void kt_mask(uint32_t (&s)[32], unsigned seen, float times)
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        s[i] = seen & (1u << i) ? __float_as_uint(__uint_as_float(s[i]) * times) : 0xFF800000u;
}

__device__ __forceinline__ float kt_max(const uint32_t (&s)[32], float top)
{
    float a = top, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        a = fmaxf(a, fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
        b = fmaxf(b, fmaxf(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])));
    }
    return fmaxf(a, b);
}

// Probabilities 2^(scale s - ref) of 32 scores as fp16 pairs; their sums are added, or put (`first`).
__device__ __forceinline__ void kt_probabilities(const uint32_t (&s)[32], f32x2 scale, f32x2 minus, bool first, f32x2 &sum, uint32_t (&p)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const f32x2 x = fma_x2(pair_x2(s[2 * i], s[2 * i + 1]), scale, minus);
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
        a = ka_exp2(a);
        b = ka_exp2(b);
        sum = first && i == 0 ? pack_x2(a, b) : kt_add_x2(sum, pack_x2(a, b));
        p[i] = ka_pack(a, b);
    }
}

// COLS columns of this thread's row times f (rare: out of line of the others).
template <int COLS>
__device__ __forceinline__ void kt_scale(uint32_t at, float f)
{
#pragma unroll 1
    for (int c = 0; c < COLS; c += 16) {
        uint32_t x[16];
        tmem_ld(at + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
        tmem_st(at + c, x);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(KtWarps<NT>::THREADS, 1) kv4_attn_tc_kernel(const KvAttnParams p)
{
    using L = KtSmem<D, NT>;
    using W = KtWarps<NT>;
    extern __shared__ __align__(1024) uint8_t kt_smem[];
    // (the same for the warp, and so that the compiler knows it)
    auto uniform = [](auto x) { return __shfl_sync(0xFFFFFFFFu, x, 0); };
    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(kt_smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(kt_smem + L::BARS);
    volatile int *flag = reinterpret_cast<volatile int *>(bars + L::COUNT);
    volatile uint32_t *slot_tm = reinterpret_cast<volatile uint32_t *>(flag + 1);
    volatile uint8_t *missing = kt_smem + L::MASK;      // of a page each
    auto bar = [&](int i) { return base + static_cast<uint32_t>(L::BARS + 8 * i); };
    const TcWait wait{flag, p.err};
    if (base & 1023u) {
        if (threadIdx.x == 0) {
            atomicOr(p.err, 4);
            pdl_wait_prior();
            p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);        // (the joining kernel goes by them)
        }
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::COUNT; ++i) {
            const bool codes = (i >= L::RAW_EMPTY && i < L::B_EMPTY);           // (RAW_EMPTY, B_FULL)
            const bool soft = (i >= L::P_FULL && i < L::O_DONE) || i >= L::Q_FULL;
            mbar_init(bar(i), i < L::RAW_EMPTY ? 2 / L::PIECES : codes ? W::CODE / 2 : soft ? W::TILE : 1);
        }
        *flag = 0;
        fence_barrier_init();
    }
    if (warp == W::MMA) {
        tmem_alloc(smem_addr(const_cast<uint32_t *>(slot_tm)), L::TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = uniform(static_cast<uint32_t>(*slot_tm));
    pdl_wait_prior();
    // (found in what the ring is later)
    static_assert(sizeof(KvPartSmem) <= L::BLOCK, "room for the parts");
    KvPart part = kv_part(p, *reinterpret_cast<KvPartSmem *>(kt_smem + L::RING));
    __syncthreads();

    // The order of an item's K and V blocks, step s of 2 n: K0 K1 V0 K2 V1 ..
    // (the scores run a unit ahead).
    struct Step {
        int unit;
        bool v;
    };
    auto step = [](int s, int n) {
        if (s == 2 * n - 1) return Step{n - 1, true};
        return s & 1 ? Step{(s + 1) >> 1, false} : s ? Step{(s >> 1) - 1, true} : Step{0, false};
    };

    if (warp == W::COPY) {
        const uint64_t policy = policy_evict_last();    // (other blocks read the same pages)
        // Four lanes, each with pages of its own: lanes 0 and 1 those of the even
        // blocks (the first conversion group's ring: K0 V0 V1 V2 ..), 2 and 3 of
        // the odd ones (K1 K2 .. and the last V).  A page is its entry's only one
        // or one of two.
        constexpr bool OWN = L::PIECES == 2;
        constexpr int PAGES = OWN ? 1 : 2;
        const int ring = (lane >> 1) & 1, sub = lane & 1, mine = OWN ? 0 : sub;
        KtTurn<L::TURN> turn;
        if (OWN && sub) turn.next();
        const long long stride = static_cast<long long>(p.kv.Hk) * kv_head_bytes(D);
        const uint32_t codes0 = base + L::RAW + ring * L::TURN * L::ENTRY + mine * (KV_PAGE * D / 2);
        const uint32_t scales0 = base + L::RAW + ring * L::TURN * L::ENTRY + PAGES * (KV_PAGE * D / 2) + mine * (KV_PAGE * D / 16);
        int units = 0;
        for (; part.left > 0; part.next(p)) {
            const KvItem &it = part.item;
            const int last = it.seq.before + kv_token(p, min((it.tile + 1) * p.tile, it.seq.n * p.G) - 1);
            if (lane == 0 && it.seq.before >= 0 && last >= p.kv.max_pages * KV_PAGE) atomicOr(p.err, KV_ERR_PAGE);
            // the item's queries on their way to L2 while the item before is at its end
            for (int r = lane; r < p.tile; r += 32) {
                const int pk = it.tile * p.tile + r, tt = kv_token(p, pk);
                if (pk < it.seq.n * p.G)
                    prefetch_l2(p.q + (it.seq.first + tt) * p.ldq + static_cast<long long>(it.h * p.G + pk - tt * p.G) * D, 2 * D);
            }
            const int n = part.n;
            // a block's page: its entry in the table, asked for a step ahead and looked at when it is needed
            if (lane < 4) {
                const int32_t *table = p.kv.table + it.b * p.kv.ldt;
                const uint8_t *head = p.kv.pages + static_cast<long long>(it.h) * kv_head_bytes(D);
                const int pages = it.seq.before < 0 ? 0 : min(last / KV_PAGE + 1, p.kv.max_pages);
                // (a unit at the window's start, or at the sinks' end, may hold a page that no row sees: it may be gone)
                const int low = p.window > 0 ? max(0, it.seq.before + kv_token(p, it.tile * p.tile) - p.window + 1) : 0;
                const int sink_pages = (min(p.sinks, low) + KV_PAGE - 1) / KV_PAGE;
                const unsigned gone = static_cast<unsigned>(max(0, low / KV_PAGE - sink_pages));
                auto seen = [&](int i) { return i < pages && static_cast<unsigned>(i - sink_pages) >= gone; };
                // the unit of step j, and whether it is of values
                auto unit = [&](int j) { return ring ? min(j + 1, n - 1) : max(j - 1, 0); };
                auto page_at = [&](int j) { return it.span.at(part.unit + unit(j)) * (KT_UNIT / KV_PAGE) + sub; };
                int at = page_at(0), id = seen(at) ? table[at] : -1;
                // and of the keys' lanes, the whole page of some units ahead on its way to L2: the ring is too short for
                // a copy from HBM
                constexpr int AHEAD = 5;
                auto far = [&](int j) { return ring && j + AHEAD < n ? it.span.at(part.unit + j + AHEAD) * (KT_UNIT / KV_PAGE) + sub : pages; };
                int at_far = far(0), id_far = at_far < pages ? table[at_far] : -1;
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    const bool v = ring ? j == n - 1 : j > 0, here = seen(at) && id >= 0 && id < p.kv.n_pages;
                    if (seen(at) && !here) atomicOr(p.err, KV_ERR_PAGE);
                    const uint8_t *src = head + id * stride;
                    const int u = unit(j);
                    at = page_at(j + 1);
                    if (j + 1 < n) id = seen(at) ? table[at] : -1;
                    if (id_far >= 0 && id_far < p.kv.n_pages) prefetch_l2(head + id_far * stride, kv_head_bytes(D));
                    at_far = far(j + 1);
                    id_far = at_far < pages ? table[at_far] : -1;
                    if (!v) missing[2 * ((units + u) & 15) + sub] = !here;
                    const int slot = ring * L::TURN + turn.at;
                    if (turn.round) wait(bar(L::RAW_EMPTY + slot), turn.round - 1);
                    const uint32_t full = bar(L::RAW_FULL + slot);
                    mbar_arrive_expect_tx(full, here ? KV_PAGE * D / 2 + KV_PAGE * D / 16 : 0);
                    if (here) {
                        bulk_g2s(codes0 + turn.at * L::ENTRY, src + (v ? kv_v_codes(D) : 0), KV_PAGE * D / 2, full, policy);
                        bulk_g2s(scales0 + turn.at * L::ENTRY, src + (v ? kv_v_scales(D) : kv_k_scales(D)), KV_PAGE * D / 16, full, policy);
                    }
                    turn.next();
                    if (OWN) turn.next();
                }
            }
            __syncwarp();
            units += n;
        }
    } else if (warp >= W::SOFT && warp < W::MMA) {
        // ------------------------------------------------ codes to fp16
        // Two groups of warps take every other block: one's waits and stores
        // overlap the other's.
        constexpr int Q32 = D / 32;             // 32-dimension pieces of a token
        constexpr int THREADS = W::CODE * 16, ROUNDS = KT_UNIT * Q32 / THREADS;
        const int group = (warp - W::SOFT) / (W::CODE / 2), me = threadIdx.x & (THREADS - 1);
        KtTurn<L::TURN> entry;
        KtTurn<L::BLOCKS> block;
        if (group) block.next();
        for (; part.left > 0; part.next(p)) {
            const int n = part.n;
#pragma unroll 1
            for (int b = group; b < 2 * n; b += 2) {    // (an item has an even number of blocks)
                const bool v = step(b, n).v;
                uint4 w[ROUNDS];
                uint32_t sc[ROUNDS];
                uint32_t free[L::PIECES];
#pragma unroll
                for (int e = 0; e < L::PIECES; ++e) {
                    const int slot = group * L::TURN + entry.at;
                    wait(bar(L::RAW_FULL + slot), entry.round);
                    const uint8_t *raw = kt_smem + L::RAW + slot * L::ENTRY;
                    constexpr int N = ROUNDS / L::PIECES;
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const int i = me + k * THREADS, row = i / Q32, q = i % Q32;
                        w[e * N + k] = *reinterpret_cast<const uint4 *>(raw + row * (D / 2) + 16 * q);
                        sc[e * N + k] = *reinterpret_cast<const uint16_t *>(raw + KT_UNIT / L::PIECES * D / 2 + row * (D / 16) + 2 * q);
                    }
                    free[e] = bar(L::RAW_EMPTY + slot);
                    entry.next();
                }
                // (the reads are done before a bulk copy may write here: without the fence it overtook them)
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int e = 0; e < L::PIECES; ++e) mbar_arrive(free[e]);
                }
                if (block.round) wait(bar(L::B_EMPTY + block.at), block.round - 1);
                const uint32_t to = base + L::RING + block.at * L::BLOCK;
#pragma unroll
                for (int k = 0; k < ROUNDS; ++k) {
                    const int i = me + k * THREADS, row = i / Q32, q = i % Q32;
                    uint32_t s2 = kv_scales2(sc[k]);
                    if (v) s2 = kv_finite2(s2);
                    // pieces of eight dimensions in an order of the thread's own, so that neighbours write
                    // different banks: piece e xor x
                    const int x = D == 64 ? 0 : D == 128 ? 2 * (q >> 1) : q >> 1;
                    uint32_t c[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                    uint32_t f[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
                    if (D == 256 && (x & 1)) {
                        const uint32_t a = c[0], b2 = c[2];
                        c[0] = c[1], c[1] = a, c[2] = c[3], c[3] = b2;
                    }
                    if (D >= 128 && (x & 2)) {
                        const uint32_t a = c[0], b2 = c[1], g = f[0];
                        c[0] = c[2], c[1] = c[3], c[2] = a, c[3] = b2;
                        f[0] = f[1], f[1] = g;
                    }
                    const uint32_t line = to + (row >> 3) * (D / 64 * 1024) + (q >> 1) * 1024 + (row & 7) * 128;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
                        kv_values8(c[e], y);
                        const int chunk = ((q & 1) * 4 + (e ^ x)) ^ (row & 7);
                        sts128(line + chunk * 16, make_uint4(kv_mul2(y[0], f[e >> 1]), kv_mul2(y[1], f[e >> 1]),
                                                             kv_mul2(y[2], f[e >> 1]), kv_mul2(y[3], f[e >> 1])));
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_FULL + block.at));
                block.next();
                block.next();
            }
        }
    } else if (warp == W::MMA) {
        // ------------------------------------------------ products
        KtTurn<L::BLOCKS> block;
        uint32_t items[NT] = {}, run[NT] = {};  // of each tile: items, units
        constexpr uint32_t GROUP = D / 64 * 1024;       // bytes of eight tokens of a block
        auto scores = [&](int tile, uint32_t s) {
            const uint64_t b0 = kt_desc(base + L::RING + block.at * L::BLOCK, 16, GROUP);
            if (NT == 1) {
#pragma unroll
                for (int k = 0; k < D / 64; ++k)
                    kt_mma4_ts_warp(tmem + s, tmem + L::QUERY + 32 * k, 0, b0 + k * (1024 >> 4), 2, kt_idesc(KT_UNIT, false), k > 0);
            } else {
                const uint64_t a0 = kt_desc(base + tile * (KT_ROWS * D * 2), 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 64; ++k)
                    kt_mma4_ss_warp(tmem + s, a0 + k * (KT_ROWS * 128 >> 4), b0 + k * (1024 >> 4), kt_idesc(KT_UNIT, false), k > 0);
            }
        };
        // (a row's first 32 probabilities are in the first 16 columns of S, the others from 32 on)
        auto values = [&](int tile, uint32_t s, bool first) {
            kt_mma4_ts_warp(tmem + L::O(tile), tmem + s, NT == 1 ? 16 : 0, kt_desc(base + L::RING + block.at * L::BLOCK, 1024, GROUP),
                            2 * GROUP >> 4, kt_idesc(D, true), !first);
        };
        auto full = [&]() {
            wait(bar(L::B_FULL + block.at), block.round);
            __syncwarp();
            tc_fence_after_sync();
        };
        auto done = [&]() {
            tc_commit_warp(bar(L::B_EMPTY + block.at));
            block.next();
        };
        for (; uniform(static_cast<int>(part.left > 0)); part.next(p)) {
            const KvItem &it = part.item;
            const int n = uniform(part.n);
            const int tiles = uniform(NT == 2 && it.seq.n * p.G - it.tile * p.tile > KT_ROWS ? 2 : 1);
            for (int t = 0; t < tiles; ++t) wait(bar(L::Q_FULL + t), t ? items[NT - 1]++ : items[0]++);
            __syncwarp();
            tc_fence_after_sync();
            // (scores go over the probabilities of the unit before the last: after their product, in order)
#pragma unroll 1
            for (int i = -1; i < n; ++i) {
                if (i + 1 < n) {
                    full();
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (t >= tiles) continue;
                        const uint32_t buf = (run[t] + (i < 0 ? 0 : 1)) & 1;
                        scores(t, L::S(t, 0) + 64 * buf);
                        tc_commit_warp(bar(L::S_FULL + 2 * t + buf));
                    }
                    done();
                }
                if (i < 0) continue;
                full();
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t >= tiles) continue;
                    const uint32_t buf = run[t] & 1;
                    wait(bar(L::P_FULL + 2 * t + buf), run[t] >> 1);
                    __syncwarp();
                    tc_fence_after_sync();
                    values(t, L::S(t, 0) + 64 * buf, i == 0);
                    tc_commit_warp(bar(L::O_DONE + 2 * t + buf));       // (two: the softmax may be that far behind)
                    ++run[t];
                }
                done();
            }
        }
    } else if (warp < W::SOFT) {
        // ------------------------------------------------ queries, softmax, outputs
        constexpr int SPLIT = 2 / NT;           // threads of a row
        const int tile = NT == 2 ? warp >> 2 : 0, group = NT == 2 ? 0 : warp >> 2, row = threadIdx.x & (KT_ROWS - 1);
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float *stat = reinterpret_cast<float *>(kt_smem + L::STAT) + row;
        float *factor = reinterpret_cast<float *>(kt_smem + L::FACTOR);
        auto together = [&]() {                 // the tile's warps
            __syncwarp();
            named_bar_sync(1 + tile, 32 * W::TILE);
        };
        uint32_t run = 0;                       // units of this thread's tile
        int units = 0;
        if (threadIdx.x == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        for (; part.left > 0; part.next(p)) {
            const KvItem &it = part.item;
            const int n = part.n, rows = min(p.tile, it.seq.n * p.G - it.tile * p.tile);
            const bool active = tile * KT_ROWS < rows;
            const int mine = tile * KT_ROWS + row, packed = it.tile * p.tile + mine;
            const bool in = mine < rows;
            const int t = kv_token(p, packed);
            // The tile's queries as fp16, each row times a power of two that brings its largest value to [2^14, 2^15),
            // and the scores' sign: copied to their places and changed there, a row by D / 8 lanes with 16 bytes each.
            if (active) {
                constexpr int LANES = D / 8, AT_ONCE = 32 / LANES, LOADS = KT_ROWS / (AT_ONCE * W::TILE), BATCH = 4;
                const int wq = warp & (W::TILE - 1), sub = lane / LANES, piece = lane % LANES;
                const unsigned peers = LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1u) << (sub * LANES);
                const uint32_t to = base + tile * (KT_ROWS * D * 2) + (piece / 8) * (KT_ROWS * 128);
                const int r0 = wq * LOADS * AT_ONCE + sub;
                auto place = [&](int r) { return to + r * 128 + (((piece % 8) ^ (r & 7)) << 4); };
                together();                     // (the outputs before have left these places)
#pragma unroll 4
                for (int i = 0; i < LOADS; ++i) {
                    const int r = r0 + i * AT_ONCE, pk = it.tile * p.tile + tile * KT_ROWS + r, tt = kv_token(p, pk);
                    const uint16_t *q = p.q + (it.seq.first + tt) * p.ldq + static_cast<long long>(it.h * p.G + pk - tt * p.G) * D;
                    if (tile * KT_ROWS + r < rows) cp_async_16(place(r), q + 8 * piece);
                }
                cp_async_commit();
                cp_async_wait_all();
#pragma unroll 1
                for (int i0 = 0; i0 < LOADS; i0 += BATCH) {
                    uint4 v[BATCH];
                    unsigned top[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int r = r0 + (i0 + i) * AT_ONCE;
                        v[i] = lds128(place(r));
                        if (tile * KT_ROWS + r >= rows) v[i] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                        top[i] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[i] = max(top[i], max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) top[i] = __reduce_max_sync(peers, top[i]);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int r = r0 + (i0 + i) * AT_ONCE, shift = xres_shift(top[i]);
                        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + shift) << 23), p.scale);
                        uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_f16x2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
                        sts128(place(r), make_uint4(w[0], w[1], w[2], w[3]));
                        // (not zero, which times the -inf of a masked score were NaN: below the smallest normal number the
                        // scores, at most 2^34 before it, are all nothing to the softmax)
                        if (piece == 0)
                            factor[tile * KT_ROWS + r] = fmaxf(fabsf(p.scale) * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23), 0x1p-126f);
                    }
                }
            }
            if (NT == 1) {                      // and this thread's part of its row to tensor memory
                together();
#pragma unroll 1
                for (int c = 0; c < D / 4; c += 16) {
                    uint32_t x[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int piece = group * (D / 16) + c / 4 + e;
                        const uint4 v = lds128(base + (piece / 8) * (KT_ROWS * 128) + row * 128 + (((piece % 8) ^ (row & 7)) << 4));
                        x[4 * e] = v.x, x[4 * e + 1] = v.y, x[4 * e + 2] = v.z, x[4 * e + 3] = v.w;
                    }
                    tmem_st(lanes + L::QUERY + group * (D / 4) + c, x);
                }
                tmem_wait_st();
                tc_fence_before_sync();
            } else {
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0 && active) mbar_arrive(bar(L::Q_FULL + tile));

            KtSight sight;
            sight.pos = in && it.seq.before >= 0 ? it.seq.before + t : -1;
            sight.low = p.window > 0 ? sight.pos - p.window + 1 : 0;
            sight.sinks = p.window > 0 ? p.sinks : 0;
            // tokens that every row of the tile sees: from .. to, and below the sinks
            const int t0 = kv_token(p, it.tile * p.tile + tile * KT_ROWS);
            const int t1 = kv_token(p, it.tile * p.tile + min(rows, (tile + 1) * KT_ROWS) - 1);
            const int to = it.seq.before < 0 ? -1 : it.seq.before + t0;
            const int from = p.window > 0 ? it.seq.before + t1 - p.window + 1 : 0;
            // (a warp's rows' factors come from other warps, which also arrive at this barrier)
            together();
            float scale = factor[tile * KT_ROWS + row], times = 1.f;
            // Scores that may pass 2^23 (queries are below 2^15 and keys 2,688 at most) are multiplied where they are masked,
            // not in the softmax's fma: there the maximum, a rounded product, and fma's exact one may be powers of two apart.
            const bool round = __any_sync(0xFFFFFFFFu, in && scale * (0x1p15f * 2688.f * D) > 0x1p23f);
            if (round) {
                times = scale;
                scale = 1.f;
            }
            float m = -INFINITY;
            f32x2 l2 = pack_x2(0.f, 0.f);
            for (int i = 0; active && i < n; ++i, ++run) {
                const uint32_t buf = run & 1;
                constexpr int CHUNKS = 2 / SPLIT;       // of 32 scores: this thread's
                const uint32_t at = lanes + L::S(tile, 0) + 64 * buf + 32 * group;
                wait(bar(L::S_FULL + 2 * tile + buf), run >> 1);
                __syncwarp();
                tc_fence_after_sync();
                uint32_t x[CHUNKS][32];
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) tmem_ld32(at + 32 * j, x[j]);
                const int first = it.span.at(part.unit + i) * KT_UNIT;
                const unsigned gone = missing[2 * ((units + i) & 15)] | missing[2 * ((units + i) & 15) + 1] << 1;
                const bool all = !gone && !round && first + KT_UNIT - 1 <= to && (first >= from || first + KT_UNIT <= sight.sinks);
                tmem_wait_ld();
                if (!all) {
#pragma unroll
                    for (int j = 0; j < CHUNKS; ++j) kt_mask(x[j], sight(first + 32 * (group + j), gone >> (group + j)), times);
                }
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) top = kt_max(x[j], top);
                if (SPLIT == 2) {               // the row's other half
                    float *of = stat + (run & 1) * (2 * KT_ROWS);       // (two of them: read before they are written again)
                    of[group * KT_ROWS] = top;
                    together();
                    top = fmaxf(top, of[(group ^ 1) * KT_ROWS]);
                }
                if (top != -INFINITY) top *= scale;
                const bool grow = top > m + KA_TOP || (m == -INFINITY && top > m);
                if (__any_sync(0xFFFFFFFFu, grow)) {
                    const float to_m = fmaxf(m, top - KA_LIFT), f = to_m == m ? 1.f : m == -INFINITY ? 0.f : ka_exp2(m - to_m);
                    m = to_m;
                    l2 = mul_x2(l2, pack_x2(f, f));
                    if (i > 0) {
                        wait(bar(L::O_DONE + 2 * tile + ((run - 1) & 1)), (run - 1) >> 1);
                        __syncwarp();
                        tc_fence_after_sync();
                        kt_scale<D / SPLIT>(lanes + L::O(tile) + group * (D / SPLIT), f);
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const f32x2 scale2 = pack_x2(scale, scale), minus = pack_x2(-ref, -ref);
                f32x2 unit2;                    // (the unit's alone first: one by one, small ones would leave a large sum as it is)
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    uint32_t pr[16];
                    kt_probabilities(x[j], scale2, minus, j == 0, unit2, pr);
                    tmem_st(at + 16 * j, pr);   // (of this thread's columns, which it has read)
                }
                l2 = kt_add_x2(l2, unit2);
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::P_FULL + 2 * tile + buf));
            }
            units += n;

            // the row's sums
            float l = sum_x2(l2);
            if (active) {
                if (SPLIT == 2) {
                    float *of = stat + 4 * KT_ROWS;
                    of[group * KT_ROWS] = l;
                    together();
                    l = of[0] + of[KT_ROWS];
                }
                wait(bar(L::O_DONE + 2 * tile + ((run - 1) & 1)), (run - 1) >> 1);
                __syncwarp();
                tc_fence_after_sync();
                const bool whole = part.whole();
                const float f = whole ? (l == 0.f ? 0.f : p.v_scale / l) : 1.f;
                constexpr int COLS = D / SPLIT;
                const int c0 = group * COLS;
                const long long slot = (2LL * blockIdx.x + (part.unit == 0)) * p.tile + mine;
                // whole rows go through the queries' place, a warp's 32 rows in its eighth, so that a store has whole
                // rows of neighbouring lanes
                constexpr int CHUNKS = COLS / 8, TURNS = CHUNKS < 8 ? CHUNKS - 1 : 7;      // 16-byte pieces of a row
                const uint32_t out = base + warp * (L::Q / W::SOFT);
#pragma unroll 1
                for (int c = 0; c < COLS; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(lanes + L::O(tile) + c0 + c, x);
                    tmem_wait_ld();
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[k] = pack_bf16x2(__uint_as_float(x[8 * e + 2 * k]) * f, __uint_as_float(x[8 * e + 2 * k + 1]) * f);
                            sts128(out + lane * (COLS * 2) + (((c / 8 + e) ^ (lane & TURNS)) << 4), make_uint4(y[0], y[1], y[2], y[3]));
                        }
                    } else if (in) {
                        uint4 *to4 = reinterpret_cast<uint4 *>(p.sums + slot * D + c0 + c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) to4[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    }
                    __syncwarp();
                }
                if (whole) {
                    const int first = tile * KT_ROWS + (warp & 3) * 32;         // the warp's rows
#pragma unroll 4
                    for (int i = lane; i < 32 * CHUNKS; i += 32) {
                        const int r = i / CHUNKS, piece = i % CHUNKS, pk = it.tile * p.tile + first + r, tt = kv_token(p, pk);
                        uint16_t *o = p.o + (it.seq.first + tt) * p.ldo + static_cast<long long>(it.h * p.G + pk - tt * p.G) * D + c0;
                        if (first + r < rows) reinterpret_cast<uint4 *>(o)[piece] = lds128(out + r * (COLS * 2) + ((piece ^ (r & TURNS)) << 4));
                    }
                }
                if (!whole && in && c0 == 0) reinterpret_cast<float2 *>(p.stats)[slot] = make_float2(m, l);
                tc_fence_before_sync();         // (O has been read: the next item's products come after Q_FULL)
            }
            if (threadIdx.x == 0 && part.parts() > 1) p.joins[blockIdx.x] = make_int4(part.parts(), it.h, it.b, it.tile);
        }
    }
    // every copy has landed and every product is done: the warps above have
    // waited for each
    pdl_launch_dependents();
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == W::MMA) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::TMEM);
    }
}

}  // namespace sv
