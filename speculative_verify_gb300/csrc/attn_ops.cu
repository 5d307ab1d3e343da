// attn_ops.cu -- the C ABI of a decoder's attention layers
// (include/specverify.h): argument checks, launch shapes and dispatch of the
// rotary, 4-bit cache and attention kernels.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "kv4_attn_tc.cuh"
#include "kv4_plan.cuh"
#include "rotary.cuh"
#include "specverify.h"
#include "sv_host.h"

namespace sv {
namespace {

constexpr int MAX_DEVICES = 64;

// The current device's facts, with the kernels' shared-memory limits raised
// once per device.
int attn_device(DeviceInfo *out)
{
    const int rc = device_info(out);
    if (rc != SV_OK) return rc;
    static std::mutex mu;
    static bool ready[MAX_DEVICES] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (ready[out->dev]) return SV_OK;
    cudaError_t e = cudaSuccess;
    auto up = [&](auto *kernel, int bytes) {
        cudaError_t r = bytes ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) : cudaSuccess;
        e = e != cudaSuccess ? e : r;
        // (else a smaller share than the blocks that fit are counted with)
        r = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        e = e != cudaSuccess ? e : r;
    };
    up(kv4_attn_kernel<64, 1>, KaShape<64, 1>::BYTES);
    up(kv4_attn_kernel<64, 2>, KaShape<64, 2>::BYTES);
    up(kv4_attn_kernel<128, 1>, KaShape<128, 1>::BYTES);
    up(kv4_attn_kernel<128, 2>, KaShape<128, 2>::BYTES);
    up(kv4_attn_kernel<256, 1>, KaShape<256, 1>::BYTES);
    up(kv4_attn_kernel<256, 2>, KaShape<256, 2>::BYTES);
    up(kv4_join_kernel<64, 1>, 0);      // (the same share: a multiprocessor changes it only when it is empty)
    up(kv4_join_kernel<64, 4>, 0);
    up(kv4_join_kernel<128, 1>, 0);
    up(kv4_join_kernel<128, 4>, 0);
    up(kv4_join_kernel<256, 1>, 0);
    up(kv4_join_kernel<256, 4>, 0);
    up(kv4_attn_tc_kernel<64, 1>, KtSmem<64, 1>::BYTES);
    up(kv4_attn_tc_kernel<64, 2>, KtSmem<64, 2>::BYTES);
    up(kv4_attn_tc_kernel<128, 1>, KtSmem<128, 1>::BYTES);
    up(kv4_attn_tc_kernel<128, 2>, KtSmem<128, 2>::BYTES);
    up(kv4_attn_tc_kernel<256, 1>, KtSmem<256, 1>::BYTES);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SV_ERR_CUDA;
    }
    ready[out->dev] = true;
    return SV_OK;
}

template <class... P, class... A>
int launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg;
    launch_config(&cfg, attr, grid, threads, smem, stream);
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}

// --------------------------------------------------------------- rotary

int check_rotary_rows(const void *x, long long ld, const void *out, long long ldo, int heads, int d)
{
    if (heads == 0) return SV_OK;
    if (!x || !out) return SV_ERR_NULL;
    if (ld < 1LL * heads * d || ldo < 1LL * heads * d) return SV_ERR_SHAPE;
    if (ld % 8 || ldo % 8 || !aligned_to(x, 16) || !aligned_to(out, 16)) return SV_ERR_ALIGN;
    return SV_OK;
}

// ---------------------------------------------------------------- cache

constexpr int KV_MAX_PAGES = 1 << 24;           // of a sequence: positions stay within 2^29

bool fine_scale(float s) { return std::isfinite(s) && s >= 1e-30f && s <= 1e30f; }

bool fine_sizes(const sv_kv4_cache *c)
{
    return (c->d == 64 || c->d == 128 || c->d == 256) && c->Hk >= 1 && c->Hk <= 65535 && c->n_pages >= 0 && c->max_pages >= 0 &&
           c->max_pages <= KV_MAX_PAGES;
}

bool fine_rows(int R, int B, bool ragged)
{
    if (R < 0 || R > (1 << 29) || B < 0 || B > (1 << 20)) return false;
    return ragged || (B ? R % B : R) == 0;      // (as many rows a sequence)
}

int check_cache(const sv_kv4_cache *c, int B)
{
    if (!c) return SV_ERR_NULL;
    if (!fine_sizes(c) || (B > 0 && c->ldt < c->max_pages)) return SV_ERR_SHAPE;
    if (!fine_scale(c->k_scale) || !fine_scale(c->v_scale)) return SV_ERR_SHAPE;
    if ((c->n_pages > 0 && !c->pages) || (B > 0 && c->max_pages > 0 && !c->page_table)) return SV_ERR_NULL;
    if (!aligned_to(c->pages, 16) || !aligned_to(c->page_table, 4)) return SV_ERR_ALIGN;
    return SV_OK;
}

int check_kv_rows(int R, const int32_t *cu, const int32_t *lens, int B)
{
    if (!fine_rows(R, B, cu)) return SV_ERR_SHAPE;
    if (B > 0 && !lens) return SV_ERR_NULL;
    if (!aligned_to(cu, 4) || !aligned_to(lens, 4)) return SV_ERR_ALIGN;
    return SV_OK;
}

KvRows kv_rows(int R, const int32_t *cu, const int32_t *lens, int B) { return KvRows{cu, lens, B, cu ? 0 : R / B, R}; }

KvPages kv_pages(const sv_kv4_cache *c)
{
    return KvPages{c->pages, c->page_table, c->ldt, c->n_pages, c->max_pages, c->Hk};
}

template <bool GATHER>
int kv_rows_call(uint16_t *k, long long ldk, uint16_t *v, long long ldv, int R, const int32_t *cu, const int32_t *lens,
                 int B, const sv_kv4_cache *c, cudaStream_t stream)
{
    int rc = check_cache(c, B);
    if (rc == SV_OK) rc = check_kv_rows(R, cu, lens, B);
    if (rc != SV_OK) return rc;
    const long long n = 1LL * c->Hk * c->d;
    if (R > 0 && (ldk < n || ldv < n)) return SV_ERR_SHAPE;
    if (R > 0 && (!k || !v)) return SV_ERR_NULL;
    if (R > 0 && (ldk % 8 || ldv % 8 || !aligned_to(k, 16) || !aligned_to(v, 16))) return SV_ERR_ALIGN;
    const long long blocks = (R * n / KV_GROUP + KV_THREADS - 1) / KV_THREADS;
    if (blocks > 0x7FFFFFFF) return SV_ERR_SHAPE;
    if (R == 0 || B == 0) return SV_OK;
    DeviceInfo dev;
    rc = attn_device(&dev);
    if (rc != SV_OK) return rc;
    const KvRowsParams p{kv_rows(R, cu, lens, B), kv_pages(c), k, v, ldk, ldv, c->k_scale, c->v_scale, dev.err};
    const dim3 grid(static_cast<unsigned>(blocks));
    switch (c->d) {
    case 64: return launch(kv4_rows_kernel<64, GATHER>, grid, KV_THREADS, 0, stream, p);
    case 128: return launch(kv4_rows_kernel<128, GATHER>, grid, KV_THREADS, 0, stream, p);
    default: return launch(kv4_rows_kernel<256, GATHER>, grid, KV_THREADS, 0, stream, p);
    }
}

// ------------------------------------------------------------ attention

// How a call's work is cut: the kernel (rows of eight of kv4_attn_kernel, or
// tiles of kv4_attn_tc_kernel), packed rows of an item, tokens of a unit, units
// that an item's start and end are counted as, parts at most, units of a part at
// least.
struct AttnPlan {
    int eights, tiles, tile, unit, extra, parts, least;
    bool joins;                                 // an item may go over several parts
    int groups;                                 // of threads of a block that joins them
};

// The parts are counted for a GPU of this size whatever the device, so that
// the workspace's size does not ask the device.
constexpr int ATTN_SMS = 152;

template <int D>
constexpr int attn_blocks(int eights) { return eights == 1 ? KaShape<D, 1>::BLOCKS : KaShape<D, 2>::BLOCKS; }

// Packed rows (a sequence's tokens times G) choose the kernel.
//   * Items of 8 rows, else 16, of kv4_attn_kernel: its time is the codes'
//     conversion, which an item has once whatever its rows, and products of rows
//     that are not there: 256 x 8 rows of 4,096 tokens (4 heads of 128) 128 us,
//     as items of 16 182.
//   * kv4_attn_tc_kernel converts once for 128 rows and more, but through
//     shared memory, and an item's start and end are long.  Against two or three
//     items of 16 rows (us, 64 sequences of 4,096 tokens, 4 heads):
//         d 64:  16 rows 40 and 103, 32 rows 66 and 104, 48 rows 93 and 105, 64 rows 118 and 108
//         d 128: 16 rows 57 and 108, 32 rows 99 and 109, 48 rows 140 and 110
//         d 256: 16 rows 89 and 143, 24 rows 160 and 144
//     and one sequence of 131,072 tokens: d 64, 48 rows 55 and 58; d 128, 32 rows
//     63 and 60, 48 rows 80 and 61; d 256, 16 rows 60 and 78, 24 rows 90 and 80.
//   * Two tiles share a unit's conversion, one tile leaves more items side by
//     side and has shorter hand-offs (us, 4 sequences of 8,192 tokens, 4 heads):
//         d 128: 256 rows 48 and 43, 384 rows 60 and 54, 512 rows 61 and 67, 2,048 rows 168 and 214
//         d 64:  128 rows 27 and 28, 192 rows 33 and 40, 512 rows 51 and 65, 2,048 rows 138 and 206
//     d 256 has room for one only.
// An item's start and end are counted as `extra` units: 8,192 rows of d 256 take
// 1,002 us with 1, 802 with 5, 742 with 10, 784 with 20.  A part is four units at
// least, a page a warp (1 row of 1,000 tokens, d 256, 11.7 us in a graph, 12.8
// with 8, 18.7 with 20).  Where items are expected in eight parts and more, four
// groups of threads join them (1 row of 16,000 tokens 26 us, 50 with one group),
// elsewhere one (nine ragged prompts 170 us, 185 with four).
// A call takes one kernel: 128 single rows of 4,096 tokens and a prompt of 2,048
// rows (4 query heads on each of 4 of 128) take 237 us together, 126 in two calls.
AttnPlan attn_plan(int R, int B, int G, int d, int Hk, int max_pages)
{
    AttnPlan a{};
    // (a sequence's, on average where they are uneven)
    const long long packed = (1LL * R * G + B - 1) / B;
    a.eights = packed <= 8 ? 1 : packed <= (d == 64 ? 48 : d == 128 ? 32 : 16) ? 2 : 0;
    a.tiles = a.eights ? 0 : d == 256 || packed <= (d == 64 ? 1 : 3) * KT_ROWS ? 1 : 2;
    a.tile = a.tiles ? a.tiles * KT_ROWS : 8 * a.eights;
    a.unit = a.tiles ? KT_UNIT : KV_PAGE;
    a.extra = a.tiles ? 10 : 4;
    a.least = 4;
    const int blocks = a.tiles ? 1 : d == 64 ? attn_blocks<64>(a.eights) : d == 128 ? attn_blocks<128>(a.eights) : attn_blocks<256>(a.eights);
    // (items, and their units, at most)
    const long long items = Hk * ((1LL * R * G + a.tile - 1) / a.tile + B);
    const long long units = items * (a.extra + std::max(1, (max_pages * KV_PAGE + a.unit - 1) / a.unit));
    a.parts = static_cast<int>(std::min<long long>(1LL * ATTN_SMS * blocks, (units + a.least - 1) / a.least));
    const long long least_items = Hk * std::max<long long>(B, (1LL * R * G + a.tile - 1) / a.tile);
    a.groups = a.parts >= 8 * least_items ? 4 : 1;
    a.joins = a.parts > 1 && max_pages * KV_PAGE > a.unit;
    return a;
}

// Workspace: joins [parts], statistics and sums of two slots a part.
struct AttnSpace {
    size_t stats, sums, bytes;
    AttnSpace(const AttnPlan &a, int d)
    {
        const size_t rows = 2 * static_cast<size_t>(a.parts) * static_cast<size_t>(a.tile);
        stats = 16 * static_cast<size_t>(a.parts);
        sums = stats + 8 * rows;
        bytes = sums + 4 * rows * static_cast<size_t>(d);
    }
};

int check_attention(int R, int B, int Hq, const sv_kv4_cache *c)
{
    if (Hq < 1 || Hq % c->Hk || 1LL * R * (Hq / c->Hk) > (1 << 29) || 1LL * R * Hq > (1LL << 33)) return SV_ERR_SHAPE;
    return SV_OK;
}

template <int D>
int attn_launch(const KvAttnParams &p, const AttnPlan &a, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(a.parts));
    int rc;
    if (a.eights == 1)
        rc = launch(kv4_attn_kernel<D, 1>, grid, KA_WARPS * 32, KaShape<D, 1>::BYTES, stream, p);
    else if (a.eights == 2)
        rc = launch(kv4_attn_kernel<D, 2>, grid, KA_WARPS * 32, KaShape<D, 2>::BYTES, stream, p);
    else if (a.tiles == 1)
        rc = launch(kv4_attn_tc_kernel<D, 1>, grid, KtWarps<1>::THREADS, KtSmem<D, 1>::BYTES, stream, p);
    else {
        if constexpr (D != 256)
            rc = launch(kv4_attn_tc_kernel<D, 2>, grid, KtWarps<2>::THREADS, KtSmem<D, 2>::BYTES, stream, p);
        else
            rc = SV_ERR_SHAPE;                  // (not planned)
    }
    if (rc != SV_OK || !a.joins) return rc;
    // (rows that an item has at most: a block without rows costs its launch all the same)
    constexpr int ROWS = KJ_VALUES / D;
    const long long rows = std::min<long long>(a.tile, 1LL * (p.rows.cu ? p.rows.R : p.rows.T) * p.G);
    const dim3 joins(static_cast<unsigned>(a.parts), static_cast<unsigned>((rows + ROWS - 1) / ROWS));
    return a.groups == 4 ? launch(kv4_join_kernel<D, 4>, joins, 4 * KJ_THREADS, 0, stream, p)
                         : launch(kv4_join_kernel<D, 1>, joins, KJ_THREADS, 0, stream, p);
}

}  // namespace
}  // namespace sv

extern "C" {

int rotary_embed(const sv_bf16 *q, long long ldq, int Hq, const sv_bf16 *k, long long ldk, int Hk, int rows, int d, int rot,
                 const int32_t *positions, long long ldp, int n_axes, const int32_t *axes, const float *inv_freq,
                 float factor, int flags, sv_bf16 *q_out, long long ldqo, sv_bf16 *k_out, long long ldko, sv_stream stream)
{
    using namespace sv;
    if (rows < 0 || rows > 1 << 30 || Hq < 0 || Hk < 0 || Hq > 65535 || Hk > 65535 || Hq + Hk < 1) return SV_ERR_SHAPE;
    if (d < 16 || d > RO_MAX_DIM || d % 8 || rot < 16 || rot > d || rot % 16) return SV_ERR_SHAPE;
    if (n_axes < 1 || n_axes > 16 || (flags & ~SV_ROTARY_PAIRED) || !std::isfinite(factor)) return SV_ERR_SHAPE;
    if (rows == 0) return SV_OK;
    int rc = check_rotary_rows(q, ldq, q_out, ldqo, Hq, d);
    if (rc == SV_OK) rc = check_rotary_rows(k, ldk, k_out, ldko, Hk, d);
    if (rc != SV_OK) return rc;
    if (!positions || !inv_freq) return SV_ERR_NULL;
    if (n_axes > 1 && ldp < rows) return SV_ERR_SHAPE;
    if (!aligned_to(positions, 4) || !aligned_to(axes, 4) || !aligned_to(inv_freq, 4)) return SV_ERR_ALIGN;
    DeviceInfo dev;
    rc = attn_device(&dev);
    if (rc != SV_OK) return rc;
    RotaryParams p{q, k, q_out, k_out, ldq, ldk, ldqo, ldko, positions, ldp, axes, inv_freq, rows, Hq, Hk, d, rot, n_axes, 1, Hq + Hk,
                   factor, dev.err};
    // a few rows: their heads over blocks, so that a thread has one item
    const int items = rot / 16 + (d - rot) / 8;
    while (p.block_rows < RO_MAX_ROWS && (rows + p.block_rows - 1) / p.block_rows > 16 * dev.sms) p.block_rows *= 2;
    if (rows < 2 * dev.sms) p.heads = std::max(1, RO_THREADS / items);
    const dim3 grid(static_cast<unsigned>((rows + p.block_rows - 1) / p.block_rows),
                    static_cast<unsigned>((Hq + Hk + p.heads - 1) / p.heads));
    const size_t smem = static_cast<size_t>(p.block_rows) * ro_place(rot / 2) * sizeof(float2);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    return flags & SV_ROTARY_PAIRED ? launch(rotary_kernel<true>, grid, RO_THREADS, smem, cs, p)
                                    : launch(rotary_kernel<false>, grid, RO_THREADS, smem, cs, p);
}

size_t kv4_page_bytes(int Hk, int d)
{
    if (Hk < 1 || Hk > 65535 || (d != 64 && d != 128 && d != 256)) return 0;
    return static_cast<size_t>(Hk) * sv::kv_head_bytes(d);
}

int kv4_append(const sv_bf16 *k, long long ldk, const sv_bf16 *v, long long ldv, int R, const int32_t *cu_seqlens,
               const int32_t *seq_lens, int B, const sv_kv4_cache *cache, sv_stream stream)
{
    return sv::kv_rows_call<false>(const_cast<sv_bf16 *>(k), ldk, const_cast<sv_bf16 *>(v), ldv, R, cu_seqlens, seq_lens, B,
                                   cache, reinterpret_cast<cudaStream_t>(stream));
}

int kv4_gather(sv_bf16 *k, long long ldk, sv_bf16 *v, long long ldv, int R, const int32_t *cu_seqlens,
               const int32_t *seq_lens, int B, const sv_kv4_cache *cache, sv_stream stream)
{
    return sv::kv_rows_call<true>(k, ldk, v, ldv, R, cu_seqlens, seq_lens, B, cache, reinterpret_cast<cudaStream_t>(stream));
}

size_t kv4_attention_bytes(int R, int B, int ragged, int Hq, const sv_kv4_cache *cache)
{
    using namespace sv;
    if (!cache || !fine_sizes(cache) || !fine_rows(R, B, ragged) || check_attention(R, B, Hq, cache) != SV_OK) return 0;
    if (R == 0 || B == 0) return 16;
    return AttnSpace(attn_plan(R, B, Hq / cache->Hk, cache->d, cache->Hk, cache->max_pages), cache->d).bytes;
}

int kv4_attention(const sv_bf16 *q, long long ldq, int R, int Hq, const int32_t *cu_seqlens, const int32_t *seq_lens, int B,
                  const sv_kv4_cache *cache, float scale, int window, int sinks, sv_bf16 *o, long long ldo, void *ws,
                  size_t ws_bytes, sv_stream stream)
{
    using namespace sv;
    int rc = check_cache(cache, B);
    if (rc == SV_OK) rc = check_kv_rows(R, cu_seqlens, seq_lens, B);
    if (rc == SV_OK) rc = check_attention(R, B, Hq, cache);
    if (rc != SV_OK) return rc;
    const long long n = 1LL * Hq * cache->d;
    // (of scores in units of log2)
    const float log_scale = static_cast<float>(static_cast<double>(scale) * cache->k_scale * 1.4426950408889634);
    if (!std::isfinite(log_scale) || window < 0 || sinks < 0 || window > (1 << 30) || sinks > (1 << 30)) return SV_ERR_SHAPE;
    if (R > 0 && (ldq < n || ldo < n)) return SV_ERR_SHAPE;
    if (R > 0 && (!q || !o)) return SV_ERR_NULL;
    if (R > 0 && (ldq % 8 || ldo % 8 || !aligned_to(q, 16) || !aligned_to(o, 16))) return SV_ERR_ALIGN;
    if (R == 0 || B == 0) return SV_OK;
    if (!ws) return SV_ERR_NULL;
    if (!aligned_to(ws, 16)) return SV_ERR_ALIGN;
    const int G = Hq / cache->Hk;
    const AttnPlan a = attn_plan(R, B, G, cache->d, cache->Hk, cache->max_pages);
    const AttnSpace at(a, cache->d);
    if (ws_bytes < at.bytes) return SV_ERR_SHAPE;
    DeviceInfo dev;
    rc = attn_device(&dev);
    if (rc != SV_OK) return rc;
    KvAttnParams p{};
    p.rows = kv_rows(R, cu_seqlens, seq_lens, B);
    p.kv = kv_pages(cache);
    p.q = q;
    p.o = o;
    p.ldq = ldq;
    p.ldo = ldo;
    p.G = G;
    p.tile = a.tile;
    for (p.tile_log = 0; 1 << p.tile_log < a.tile; ++p.tile_log) {}
    for (p.unit_log = 0; 1 << p.unit_log < a.unit; ++p.unit_log) {}
    unsigned c = 0;
    while (1 << c < G) ++c;
    p.g_shift = 30 + c;
    p.g_mul = static_cast<unsigned>(((1ull << p.g_shift) + static_cast<unsigned>(G) - 1) / static_cast<unsigned>(G));
    p.scale = log_scale;
    p.v_scale = cache->v_scale;
    p.window = window;
    p.sinks = sinks;
    p.extra = a.extra;
    p.least = a.least;
    p.joins = static_cast<int4 *>(ws);
    p.stats = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + at.stats);
    p.sums = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + at.sums);
    p.err = dev.err;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    switch (cache->d) {
    case 64: return attn_launch<64>(p, a, cs);
    case 128: return attn_launch<128>(p, a, cs);
    default: return attn_launch<256>(p, a, cs);
    }
}

}  // extern "C"
