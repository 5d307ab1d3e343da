// kv4.cuh -- a key and value cache held in 4 bits: its format, the rows of a
// call, and the kernels that append rows to it and read them back.
//
// A page holds 32 tokens of every key/value head, a head's part in one piece
// of 36 d bytes (one bulk copy): K codes [32][d / 2], V codes [32][d / 2], K
// scales [32][d / 16], V scales [32][d / 16].  A code is an e2m1 number, the
// even dimension in the low half of its byte; a scale is an e4m3 number for 16
// dimensions of a token, so a value takes 4.5 bits:
//     value = e2m1(code) * e4m3(scale) * g,   g the tensor's k_scale or v_scale.
// e2m1 * e4m3 has six significant bits and is exact in fp16 (2^-10 .. 2,688),
// which is what the attention kernels multiply.
//
// Appending: scale = e4m3(max|x| / 6 g), code = e2m1(x / (g scale)), both to
// the nearest, ties to even, quotients in fp32 with IEEE division.  16
// dimensions that hold a NaN or an infinity get a NaN scale; the first scale
// of K is then NaN too, whichever of K and V it was: the attention kernels
// take a token's scores, not its values, as the sign that it is not a number
// (a masked token's values meet a probability of zero, and zero times NaN
// would reach rows that do not see it).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "sv_ptx.cuh"

namespace sv {

constexpr int KV_PAGE = 32;                     // tokens of a page
constexpr int KV_GROUP = 16;                    // dimensions of a scale
constexpr int KV_ERR_SEQLENS = 0x10;            // SV_DEVERR_BAD_SEQLENS
constexpr int KV_ERR_PAGE = 0x20;               // SV_DEVERR_BAD_PAGE
constexpr int KV_THREADS = 128;

__host__ __device__ constexpr int kv_head_bytes(int d) { return 36 * d; }
__host__ __device__ constexpr int kv_v_codes(int d) { return 16 * d; }
__host__ __device__ constexpr int kv_k_scales(int d) { return 32 * d; }
__host__ __device__ constexpr int kv_v_scales(int d) { return 34 * d; }

// Where a call's rows belong: sequence b has rows cu[b] .. cu[b + 1] (clamped
// to 0 .. R), or T each without cu; its first row has position lens[b].
struct KvRows {
    const int32_t *cu, *lens;
    int B, T, R;

    __device__ __forceinline__ void range(int b, int &first, int &end) const
    {
        if (!cu) {
            first = b * T;
            end = first + T;
            return;
        }
        first = min(max(cu[b], 0), R);
        end = max(min(max(cu[b + 1], 0), R), first);
    }
};

struct KvPages {
    uint8_t *pages;                             // [n_pages][Hk][36 d]
    const int32_t *table;                       // [B][max_pages], ldt apart
    long long ldt;
    int n_pages, max_pages, Hk;

    // The page that holds a sequence's tokens 32 i .. 32 i + 31; -1: none.
    __device__ __forceinline__ int at(int b, int i) const { return i < 0 || i >= max_pages ? -1 : page(table[b * ldt + i]); }
    // A table's entry as a page; -1: none.
    __device__ __forceinline__ int page(int id) const { return id >= 0 && id < n_pages ? id : -1; }
    template <int D>
    __device__ __forceinline__ uint8_t *head(int page, int h) const
    {
        return pages + (static_cast<long long>(page) * Hk + h) * kv_head_bytes(D);
    }
};

// Row r's sequence and position; false for a row of no sequence.
__device__ __forceinline__ bool kv_place(const KvRows &w, int r, int &b, int &pos)
{
    if (!w.cu) {
        b = r / w.T;
        const int len = w.lens[b];
        pos = len < 0 ? -1 : len > 0x3FFFFFFF ? 0x7FFFFFFF : len + r - b * w.T;
        return true;
    }
    int lo = 0, hi = w.B;                       // the last b with cu[b] <= r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (w.cu[mid] <= r) lo = mid;
        else hi = mid;
    }
    b = lo;
    const int first = w.cu[b];
    if (first > r || w.cu[b + 1] <= r || first < 0) return false;
    const int len = w.lens[b];
    pos = len < 0 ? -1 : len > 0x3FFFFFFF ? 0x7FFFFFFF : len + r - first;
    return true;
}

// One value pair's codes, x / s to the nearest e2m1, and back.
__device__ __forceinline__ uint32_t kv_code2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u32.u8 %0, c;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The four code pairs of a word as fp16 pairs, low byte first.
__device__ __forceinline__ void kv_values8(uint32_t w, uint32_t (&v)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(w));
}

// Two scales (the low 16 bits) as an fp16 pair.
__device__ __forceinline__ uint32_t kv_scales2(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
    return r;
}

__device__ __forceinline__ uint32_t kv_mul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A scale that is not a number as the largest one.
__device__ __forceinline__ uint32_t kv_finite2(uint32_t a)
{
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x5F005F00u));     // 448
    return r;
}

struct KvRowsParams {
    KvRows rows;
    KvPages kv;
    uint16_t *k, *v;                            // [R][Hk][d] (read by append, written by gather)
    long long ldk, ldv;
    float k_scale, v_scale;
    int *err;
};

// 16 values to a scale byte and eight code bytes; `bad`: they hold a NaN or an infinity.
__device__ __forceinline__ uint2 kv_quantise(const uint4 (&x)[2], float g, uint32_t &scale, bool &bad)
{
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t top = 0;                           // the largest magnitude's bits
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    bad = top >= 0x7F80u;
    const float a = __uint_as_float(top << 16), want = fminf(__fdiv_rn(a, 6.f * g), 448.f);
    uint16_t s2;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(want));
    scale = bad ? 0x7Fu : s2 & 0xFFu;
    uint32_t h = kv_scales2(scale);
    float s;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(s) : "r"(h));
    s *= g;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = kv_code2(__fdiv_rn(__uint_as_float(w[i] << 16), s), __fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), s));
    if (bad || !(s > 0.f)) return make_uint2(0u, 0u);
    return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// 16 values of eight code bytes and a scale byte, as bf16.
__device__ __forceinline__ void kv_restore(uint2 codes, uint32_t scale, float g, uint4 (&x)[2])
{
    const uint32_t h = kv_scales2(scale | scale << 8);
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t v[4];
        kv_values8(i ? codes.y : codes.x, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                : "=f"(lo), "=f"(hi) : "r"(kv_mul2(v[j], h)));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[4 * i + j]) : "f"(hi * g), "f"(lo * g));
        }
    }
    x[0] = make_uint4(out[0], out[1], out[2], out[3]);
    x[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// A thread takes 16 dimensions of K and of V of a row and head.  GATHER reads
// them back instead (zeros where the sequence is inactive or has no page).
// Appending 4,817 ragged rows of 8 heads of 128 and reading them back takes
// 18.3 us, 2.8 TB/s: the chain place - table - rows of a thread, and 32 IEEE
// divisions (with quotients by an estimate and its remainder 16.8).  32 rows take
// 5.6 us for the two calls in a graph.
template <int D, bool GATHER>
__global__ void __launch_bounds__(KV_THREADS) kv4_rows_kernel(const KvRowsParams p)
{
    constexpr int N = D / KV_GROUP;             // threads of a row and head
    pdl_launch_dependents();
    pdl_wait_prior();
    const long long i = static_cast<long long>(blockIdx.x) * KV_THREADS + threadIdx.x, rh = i / N;
    const int g = static_cast<int>(i % N);
    const bool in = rh < static_cast<long long>(p.rows.R) * p.kv.Hk;
    const int r = in ? static_cast<int>(rh / p.kv.Hk) : 0, h = static_cast<int>(rh % p.kv.Hk);
    int b = 0, pos = -1;
    const bool mine = in && kv_place(p.rows, r, b, pos);
    const int page = mine && pos >= 0 ? p.kv.at(b, pos / KV_PAGE) : -1;
    if (mine && pos >= 0 && page < 0) atomicOr(p.err, KV_ERR_PAGE);
    uint8_t *head = page >= 0 ? p.kv.head<D>(page, h) : nullptr;
    const int t = pos % KV_PAGE;
    uint4 *kp = reinterpret_cast<uint4 *>(p.k + r * p.ldk + h * D + KV_GROUP * g);
    uint4 *vp = reinterpret_cast<uint4 *>(p.v + r * p.ldv + h * D + KV_GROUP * g);
    if constexpr (GATHER) {
        if (!mine) return;
        uint4 k[2] = {}, v[2] = {};
        if (head) {
            kv_restore(*reinterpret_cast<const uint2 *>(head + t * (D / 2) + 8 * g), head[kv_k_scales(D) + t * N + g], p.k_scale, k);
            kv_restore(*reinterpret_cast<const uint2 *>(head + kv_v_codes(D) + t * (D / 2) + 8 * g),
                       head[kv_v_scales(D) + t * N + g], p.v_scale, v);
        }
        kp[0] = k[0];
        kp[1] = k[1];
        vp[0] = v[0];
        vp[1] = v[1];
    } else {
        uint32_t ks = 0, vs = 0;
        uint2 kc{}, vc{};
        bool kbad = false, vbad = false;
        if (head) {
            const uint4 k[2] = {kp[0], kp[1]}, v[2] = {vp[0], vp[1]};
            kc = kv_quantise(k, p.k_scale, ks, kbad);
            vc = kv_quantise(v, p.v_scale, vs, vbad);
        }
        // (a row and head's N threads are neighbours in a warp)
        const unsigned any = __ballot_sync(0xFFFFFFFFu, kbad || vbad);
        if (!head) return;
        const unsigned mask = (N == 32 ? 0xFFFFFFFFu : (1u << N) - 1u) << (threadIdx.x & 31 & ~(N - 1));
        if (g == 0 && (any & mask)) ks = 0x7Fu;
        *reinterpret_cast<uint2 *>(head + t * (D / 2) + 8 * g) = kc;
        *reinterpret_cast<uint2 *>(head + kv_v_codes(D) + t * (D / 2) + 8 * g) = vc;
        head[kv_k_scales(D) + t * N + g] = static_cast<uint8_t>(ks);
        head[kv_v_scales(D) + t * N + g] = static_cast<uint8_t>(vs);
    }
}

}  // namespace sv
