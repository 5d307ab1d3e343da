// rotary.cuh -- rotary positions into rows of queries and keys: pair i of a
// head turns by positions[axes[i]][row] * inv_freq[i], one axis or several
// (time, height and width of a video, say), the whole head or its first `rot`
// dimensions.
//
// Far positions: position * frequency in fp32 is off by 2^-24 of an angle of
// up to a million radians.  A frequency is instead taken once as a fraction of
// a turn in 64-bit fixed point (from its product with 1 / 2 pi in fp64), and
// the position multiplies it as an integer: whole turns drop off the top.  For
// frequencies up to 1 a step the product is within 2^-24 of a turn for every
// 32-bit position, 2^-35 for those below a million.  cos and sin are then of an
// angle of half a turn at most, as an fp32 number: 2^-26 of a turn more.
//
// The rotation is fp32 and rounded once to bf16.  Each value is read and
// written once, 16 bytes at a time; a thread block computes its rows' angles
// once for all their heads.  Bound by HBM: 8,192 rows of 32 + 8 heads of 128
// with three axes take 29.4 us, 5.7 TB/s; several items in flight in a thread
// and blocks of 512 threads (30.9 us) or 128 (34.5) were slower.  One row is at
// its launch (2.0 us in a graph).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "sv_ptx.cuh"

namespace sv {

constexpr int RO_THREADS = 256;
constexpr int RO_MAX_ROWS = 8;                  // rows of a block
constexpr int RO_MAX_DIM = 1024;
constexpr int RO_ERR_AXIS = 0x40;               // SV_DEVERR_BAD_AXIS

struct RotaryParams {
    const uint16_t *q, *k;                      // [rows][Hq][d], [rows][Hk][d]
    uint16_t *q_out, *k_out;
    long long ldq, ldk, ldqo, ldko;
    const int32_t *positions;                   // [n_axes][rows], ldp apart
    long long ldp;
    const int32_t *axes;                        // [rot / 2], or null: axis 0
    const float *inv_freq;                      // [rot / 2]
    int rows, Hq, Hk, d, rot, n_axes;
    int block_rows, heads;                      // rows of a block, heads of a block (of Hq + Hk)
    float factor;
    int *err;
};

// Places of a row's angles in shared memory, eight and two to spare: threads
// that read eight each, 80 bytes apart, meet no bank conflict.
__host__ __device__ constexpr int ro_place(int j) { return (j >> 3) * 10 + (j & 7); }

// cos and sin of `pos` steps of frequency f, times the factor.
__device__ __forceinline__ float2 ro_turn(float f, int pos, float factor)
{
    double turns = static_cast<double>(f) * 0.15915494309189533577;    // 1 / 2 pi
    turns -= rint(turns);
    const long long step = __double2ll_rn(turns * 18446744073709551616.0);     // 2^64 steps a turn
    const long long at = static_cast<long long>(static_cast<unsigned long long>(step) * static_cast<unsigned long long>(static_cast<long long>(pos)));
    float s, c;
    // (an infinite or NaN frequency: NaN, as the formula gives)
    sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 0x1p-31f + (f - f), &s, &c);
    return make_float2(c * factor, s * factor);
}

__device__ __forceinline__ void ro_pair(float2 cs, float a, float b, float &x, float &y)
{
    x = fmaf(a, cs.x, -(b * cs.y));
    y = fmaf(b, cs.x, a * cs.y);
}

__device__ __forceinline__ uint32_t ro_pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float ro_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float ro_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// PAIRED: pairs are neighbours (2i, 2i + 1); else halves apart (i, i + rot / 2).
template <bool PAIRED>
__global__ void __launch_bounds__(RO_THREADS) rotary_kernel(const RotaryParams p)
{
    extern __shared__ __align__(16) float2 ro_cs[];     // [block_rows][ro_place(rot / 2)]
    const int half = p.rot / 2, wide = ro_place(half), row0 = static_cast<int>(blockIdx.x) * p.block_rows;
    const int rows = min(p.block_rows, p.rows - row0);
    pdl_launch_dependents();
    pdl_wait_prior();
    for (int i = threadIdx.x; i < rows * half; i += RO_THREADS) {
        const int r = i / half, j = i - r * half;
        int axis = p.axes ? p.axes[j] : 0;
        if (axis < 0 || axis >= p.n_axes) {
            atomicOr(p.err, RO_ERR_AXIS);
            axis = 0;
        }
        ro_cs[r * wide + ro_place(j)] = ro_turn(p.inv_freq[j], p.positions[axis * p.ldp + row0 + r], p.factor);
    }
    __syncthreads();
    // a thread's item: 8 pairs of a head (two 16-byte pieces), or 16 bytes past the rotated part
    const int turned = p.rot / 16, items = turned + (p.d - p.rot) / 8;
    const int h0 = static_cast<int>(blockIdx.y) * p.heads, nh = min(p.heads, p.Hq + p.Hk - h0);
    for (int i = threadIdx.x; i < rows * nh * items; i += RO_THREADS) {
        const int rh = i / items, it = i - rh * items, r = rh / nh, h = h0 + rh - r * nh;
        const bool key = h >= p.Hq;
        const uint16_t *in = key ? p.k + (row0 + r) * p.ldk + static_cast<long long>(h - p.Hq) * p.d
                                 : p.q + (row0 + r) * p.ldq + static_cast<long long>(h) * p.d;
        uint16_t *out = key ? p.k_out + (row0 + r) * p.ldko + static_cast<long long>(h - p.Hq) * p.d
                            : p.q_out + (row0 + r) * p.ldqo + static_cast<long long>(h) * p.d;
        if (it >= turned) {
            if (in == out) continue;
            const int at = p.rot + 8 * (it - turned);
            *reinterpret_cast<uint4 *>(out + at) = *reinterpret_cast<const uint4 *>(in + at);
            continue;
        }
        const int a0 = PAIRED ? 16 * it : 8 * it, b0 = PAIRED ? a0 + 8 : a0 + half;
        const uint4 a = *reinterpret_cast<const uint4 *>(in + a0), b = *reinterpret_cast<const uint4 *>(in + b0);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
        uint32_t x[4], y[4];
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 two = reinterpret_cast<const float4 *>(ro_cs + r * wide + 10 * it)[j];
            cs[2 * j] = make_float2(two.x, two.y);
            cs[2 * j + 1] = make_float2(two.z, two.w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float s0, s1, t0, t1;
            if (PAIRED) {
                ro_pair(cs[j], ro_lo(u[j]), ro_hi(u[j]), s0, s1);
                ro_pair(cs[j + 4], ro_lo(v[j]), ro_hi(v[j]), t0, t1);
            } else {
                ro_pair(cs[2 * j], ro_lo(u[j]), ro_lo(v[j]), s0, t0);
                ro_pair(cs[2 * j + 1], ro_hi(u[j]), ro_hi(v[j]), s1, t1);
            }
            x[j] = ro_pack(s0, s1);
            y[j] = ro_pack(t0, t1);
        }
        *reinterpret_cast<uint4 *>(out + a0) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4 *>(out + b0) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

}  // namespace sv
