// kv4_plan.cuh -- how the attention kernels share out their work, and the
// kernel that joins what they leave in parts.
//
// Query rows are packed: row r of a sequence and key/value head is token
// r / G, query head r % G of the head's G.  An item is a tile of packed rows of
// one head; its units are the pages, or pairs of them, that some row of the
// tile sees (those of the first tokens, then those of the window).  The items
// of head 0, then head 1 and so on make one line of units, cut into equal parts,
// one for a thread block: uneven sequences and triangles of prompts cost no
// balance, and one long sequence is spread over the whole GPU.  An item's start and end cost
// as much as some units (`extra`): it is that much longer on the line, and a part
// that ends there leaves it to the next.
//
// A block whose part holds an item whole writes its outputs; of an item that
// goes on into other parts each block leaves its sums, unnormalised, with
// their maximum: the block where the item starts in its slot 1, the others in
// their slot 0.  kv4_join_kernel adds them in an order that is fixed, so results
// are the same every time.  Nothing has to be cleared first and no atomic is
// involved: calls with workspaces of their own may overlap, in graphs too.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kv4.cuh"

namespace sv {

struct KvAttnParams {
    KvRows rows;
    KvPages kv;
    const uint16_t *q;
    uint16_t *o;
    long long ldq, ldo;
    int G;                                      // query heads of a key/value head
    unsigned g_mul, g_shift;                    // r / G = r g_mul >> g_shift for r < 2^30
    int tile, tile_log;                         // packed rows of an item, a power of two
    int unit_log;                               // log2 of the tokens of a unit
    float scale;                                // of scores, with k_scale and log2 e
    float v_scale;
    int window, sinks;                          // 0: no window
    int extra;                                  // what an item takes besides its units, in units
    int least;                                  // units of a part at least
    float *sums, *stats;                        // [2 parts][tile][d], [2 parts][tile][2]
    int4 *joins;                                // [parts]
    int *err;
};

// The token of a packed row.
__device__ __forceinline__ int kv_token(const KvAttnParams &p, int r)
{
    return static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(r)) * p.g_mul >> p.g_shift);
}

// The largest position of a sequence's first row: with 2^29 rows at most no
// position passes 31 bits, and a window of 2^30 at most has left the 2^29 tokens
// that a table may have, as it has for any position beyond.
constexpr int KP_MAX_BEFORE = (1 << 30) + (1 << 29) - 1;

// A sequence's rows, and the position of its first one (negative: inactive).
struct KvSeq {
    int first, n, before;
};

__device__ __forceinline__ KvSeq kv_seq(const KvAttnParams &p, int b)
{
    KvSeq s;
    int end;
    p.rows.range(b, s.first, end);
    s.n = end - s.first;
    s.before = min(p.rows.lens[b], KP_MAX_BEFORE);
    return s;
}

// A tile's visible units of tokens: 0 .. sinks - 1, then from .. to - 1.
struct KvSpan {
    int sinks, from, to;
    __device__ __forceinline__ int units() const { return max(1, sinks + to - from); }
    __device__ __forceinline__ int at(int u) const { return u < sinks ? u : from + u - sinks; }
};

__device__ __forceinline__ int kv_tiles(const KvAttnParams &p, const KvSeq &s) { return (s.n * p.G + p.tile - 1) >> p.tile_log; }

__device__ __forceinline__ KvSpan kv_span(const KvAttnParams &p, const KvSeq &s, int tile)
{
    if (s.before < 0) return KvSpan{0, 0, 0};   // (one unit of no tokens)
    const int t0 = kv_token(p, tile * p.tile), t1 = kv_token(p, min((tile + 1) * p.tile, s.n * p.G) - 1);
    const int lo = p.window > 0 ? max(0, s.before + t0 - p.window + 1) : 0;
    const int to = (min(s.before + t1, p.kv.max_pages * KV_PAGE - 1) >> p.unit_log) + 1;
    const int sinks = min((min(p.sinks, lo) + (1 << p.unit_log) - 1) >> p.unit_log, to);
    return KvSpan{sinks, min(max(sinks, lo >> p.unit_log), to), to};
}

// An item, and a place on the line that is its.
struct KvItem {
    int h, b, tile, place;
    KvSeq seq;
    KvSpan span;
};

// Length of the line of one head's items of the 32 sequences from b0 on, and
// their rows (whole warps call it); with `want` >= 0 also the item that has place
// `want` of it.
__device__ __forceinline__ long long kv_group(const KvAttnParams &p, int b0, long long want, KvItem *found, long long &rows)
{
    const int lane = threadIdx.x & 31;
    const KvSeq mine = b0 + lane < p.rows.B ? kv_seq(p, b0 + lane) : KvSeq{};
    const int tiles = kv_tiles(p, mine);
    rows = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(mine.n) & 0xFFFFu) +
           (static_cast<long long>(__reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(mine.n) >> 16)) << 16);
    // sequences side by side, or one after another with their tiles over the
    // lanes, whichever takes fewer rounds
    const unsigned many = (static_cast<unsigned>(tiles) + 31u) >> 5;
    const bool one = __reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(tiles)) > __reduce_add_sync(0xFFFFFFFFu, min(many, 1u << 24));
    long long total = 0;
    for (int s = 0; s < (one ? 32 : 1); ++s) {
        KvSeq seq = mine;
        int n = 1;                              // rounds
        if (one) {
            seq.first = __shfl_sync(0xFFFFFFFFu, mine.first, s);
            seq.n = __shfl_sync(0xFFFFFFFFu, mine.n, s);
            seq.before = __shfl_sync(0xFFFFFFFFu, mine.before, s);
            n = (kv_tiles(p, seq) + 31) / 32;
        }
        for (int k = 0; k < n; ++k) {
            long long units = 0;
            if (one) {
                const int t = 32 * k + lane;
                if (t < kv_tiles(p, seq)) units = p.extra + kv_span(p, seq, t).units();
            } else {
                for (int t = 0; t < tiles; ++t) units += p.extra + kv_span(p, seq, t).units();
            }
            long long run = units;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long below = __shfl_up_sync(0xFFFFFFFFu, run, o);
                if (lane >= o) run += below;
            }
            const unsigned past = want >= 0 ? __ballot_sync(0xFFFFFFFFu, total + run > want) : 0u;
            if (past) {
                const int w = __ffs(past) - 1;
                long long rest = want - total - __shfl_sync(0xFFFFFFFFu, run - units, w);
                found->b = one ? b0 + s : b0 + w;
                found->seq.first = __shfl_sync(0xFFFFFFFFu, seq.first, w);
                found->seq.n = __shfl_sync(0xFFFFFFFFu, seq.n, w);
                found->seq.before = __shfl_sync(0xFFFFFFFFu, seq.before, w);
                found->tile = one ? 32 * k + w : 0;
                found->span = kv_span(p, found->seq, found->tile);
                while (rest >= p.extra + found->span.units()) {
                    rest -= p.extra + found->span.units();
                    found->span = kv_span(p, found->seq, ++found->tile);
                }
                found->place = static_cast<int>(rest);
                return total;
            }
            total += __shfl_sync(0xFFFFFFFFu, run, 31);
        }
    }
    return total;
}

// A block's part of the line: what is left of it, and the item that it is in,
// of which it has n > 0 units from `unit` on.
struct KvPart {
    long long left, share;
    int unit, n;
    KvItem item;

    // The item's units in this part.
    __device__ __forceinline__ void enter(const KvAttnParams &p)
    {
        const long long end = min(item.place + left, static_cast<long long>(p.extra + item.span.units()));
        unit = max(0, item.place - p.extra);
        n = max(0, static_cast<int>(end) - p.extra) - unit;
        if (n <= 0) left = 0;                   // (it ends with the item's start)
    }

    // Part k of `parts`, by one whole warp.  unit[g] and rows[g] are those of
    // group g of `groups`, or null: there are too many, and it goes through all.
    __device__ __forceinline__ void find(const KvAttnParams &p, int k, int parts, const long long *unit, const long long *rows, int groups)
    {
        const int lane = threadIdx.x & 31;
        left = 0;
        share = 1;
        long long line = 0, n = 0;
        if (unit) {
            for (int g = lane; g < groups; g += 32) {
                line += unit[g];
                n += rows[g];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                line += __shfl_xor_sync(0xFFFFFFFFu, line, o);
                n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
            }
        } else {
            for (int b0 = 0; b0 < p.rows.B; b0 += 32) {
                long long r;
                line += kv_group(p, b0, -1, nullptr, r);
                n += r;
            }
        }
        if (n > p.rows.R) {                     // cu_seqlens that decrease
            if (lane == 0) atomicOr(p.err, KV_ERR_SEQLENS);
            return;
        }
        if (line == 0) return;
        const long long all = line * p.kv.Hk;
        share = max(static_cast<long long>(p.least), (all + parts - 1) / parts);
        const long long lo = min(share * k, all);
        if (lo == all) return;
        item.h = static_cast<int>(lo / line);
        item.b = -1;
        long long at = lo - item.h * line, r;
        for (int b0 = 0; b0 < p.rows.B && item.b < 0; b0 += 32) {
            if (unit && at >= unit[b0 >> 5]) {
                at -= unit[b0 >> 5];
                continue;
            }
            at -= kv_group(p, b0, at, &item, r);
        }
        if (item.b < 0) return;                 // (lengths were written meanwhile)
        left = min(share, all - lo);
        enter(p);
    }
    // To the next item.
    __device__ __forceinline__ void next(const KvAttnParams &p)
    {
        left -= p.extra + unit + n - item.place;
        if (left <= 0) return;
        item.place = 0;
        if (++item.tile >= kv_tiles(p, item.seq)) {
            item.tile = 0;
            do {
                if (++item.b == p.rows.B) {
                    item.b = 0;
                    if (++item.h == p.kv.Hk) {  // (lengths written meanwhile)
                        left = 0;
                        return;
                    }
                }
                item.seq = kv_seq(p, item.b);
            } while (item.seq.n <= 0);
        }
        item.span = kv_span(p, item.seq, item.tile);
        enter(p);
    }
    __device__ __forceinline__ bool whole() const { return unit == 0 && n == item.span.units(); }
    // Whether the item starts here, and goes on in this many parts in all.
    __device__ __forceinline__ int parts() const
    {
        return unit ? 0 : 1 + static_cast<int>((item.span.units() - n + share - 1) / share);
    }
};

// The block's part, found by all its warps (all its threads call it).
constexpr int KP_GROUPS = 64;                   // of 32 sequences, that the warps share out

struct KvPartSmem {
    long long unit[KP_GROUPS], rows[KP_GROUPS];
    KvPart part;
};

__device__ __forceinline__ KvPart kv_part(const KvAttnParams &p, KvPartSmem &sm)
{
    const int groups = (p.rows.B + 31) >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool shared = groups <= KP_GROUPS;
    if (shared) {
        for (int g = warp; g < groups; g += static_cast<int>(blockDim.x >> 5)) {
            long long rows;
            const long long units = kv_group(p, 32 * g, -1, nullptr, rows);
            if (lane == 0) {
                sm.unit[g] = units;
                sm.rows[g] = rows;
            }
        }
        __syncwarp();
        __syncthreads();
    }
    if (warp == 0) {
        KvPart part{};
        part.find(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), shared ? sm.unit : nullptr, sm.rows, groups);
        if (lane == 0) sm.part = part;
        __syncwarp();
    }
    __syncthreads();
    return sm.part;
}

constexpr int KJ_VALUES = 512;                  // output values of a block, four of a thread
constexpr int KJ_THREADS = KJ_VALUES / 4;       // of a group
constexpr int KJ_MAX_PARTS = 1024;

// Block (p, s): values s KJ_VALUES .. of the item that starts in part p and
// goes on, joined from its parts.  What bounds it is the chain of loads over
// the parts: hence eight loads at a time, and where the parts are many GROUPS
// of threads that share them out.
template <int D, int GROUPS>
__global__ void __launch_bounds__(GROUPS *KJ_THREADS) kv4_join_kernel(const KvAttnParams p)
{
    constexpr int ROWS = KJ_VALUES / D;
    __shared__ float weight[ROWS][KJ_MAX_PARTS];
    __shared__ float norm[ROWS];
    __shared__ float4 others[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? KJ_THREADS : 1];    // (not the first group's)
    pdl_wait_prior();                           // (without an early start of the next kernel: it cost an attention 70 of 190 us)
    const int part = blockIdx.x, row0 = blockIdx.y * ROWS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 join = p.joins[part];            // parts; head, sequence, tile
    if (join.x < 2 || join.x > KJ_MAX_PARTS) return;
    const KvSeq seq = kv_seq(p, join.z);
    const int rows = min(p.tile, seq.n * p.G - join.w * p.tile), n = join.x;
    if (row0 >= rows) return;
    auto slot = [&](int i) { return static_cast<long long>(2 * (part + i) + (i == 0)) * p.tile; };
    for (int r = warp; r < ROWS; r += GROUPS * KJ_THREADS / 32) {
        if (row0 + r >= rows) continue;
        const float2 *stats = reinterpret_cast<const float2 *>(p.stats) + row0 + r;
        float top = -INFINITY;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(stats + slot(i)).x);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (top == -INFINITY) top = 0.f;
        float total = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float2 s = __ldcg(stats + slot(i));
            const float w = exp2f(s.x - top);
            weight[r][i] = w;
            total += w * s.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        if (lane == 0) norm[r] = total == 0.f ? 0.f : p.v_scale / total;
    }
    __syncthreads();
    const int group = threadIdx.x / KJ_THREADS, value = threadIdx.x % KJ_THREADS;
    const int r = 4 * value / D, d = 4 * value % D, row = row0 + r;
    const bool in = row < rows;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *sums = p.sums + static_cast<long long>(row) * D + d;
#pragma unroll 8
    for (int i = group; i < n && in; i += GROUPS) {
        const float4 v = ldcg_f4(sums + slot(i) * D);
        const float w = weight[r][i];
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
    }
    if (GROUPS > 1) {
        if (group) others[group][value] = acc;
        __syncthreads();
#pragma unroll
        for (int k = 1; k < GROUPS; ++k) {
            const float4 v = others[k][value];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
    }
    if (group || !in) return;
    const int packed = join.w * p.tile + row, t = kv_token(p, packed), g = packed - t * p.G;
    uint16_t *o = p.o + (seq.first + t) * p.ldo + static_cast<long long>(join.y * p.G + g) * D + d;
    const float f = norm[r];
    uint2 out;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out.x) : "f"(acc.y * f), "f"(acc.x * f));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out.y) : "f"(acc.w * f), "f"(acc.z * f));
    *reinterpret_cast<uint2 *>(o) = out;
}

}  // namespace sv
