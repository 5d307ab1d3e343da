// rmsnorm.cuh -- residual addition and root-mean-square norm of rows, with a
// bf16 or an 8-bit (e4m3 with fp32 scales) output.
//
//   s = bf16(x + r)                      (s = x without a residual)
//   y = s / sqrt(mean(s^2) + eps) * w    (or * (1 + w))
//   8 bits: scale = max|y| / 448 over 128 columns or the row, q = e4m3(y / scale)
//
// The row's norm cancels from y / scale: with z = s w, exact in fp32 (two
// bf16 factors; z = s (1 + w) is rounded twice), q = e4m3(448 z / max|z|) has
// one more rounding before its own.
//
// One block per row, the row held in registers (as bf16) between the sum of squares
// and the output, so that every byte crosses memory once: the kernel is
// bound by HBM for long inputs and by its launch and one memory round trip
// for a few rows.  VEC columns per access: 8 (16 bytes) where the row length,
// the strides and the addresses allow it, or are off by as much in every
// tensor; else 1.  Sums, the norm and the scales are fp32; the
// only roundings to fewer bits are s (the value that the next layer adds to,
// as the residual stream is kept in bf16) and the output's.  Long rows do not
// fit 64 registers a thread whole: of those beyond 32,768 columns 100 to 280
// bytes a thread are in local memory, of those that go column by column
// beyond 8,192 40 to 160, beyond 16,384 2 to 3 KB (L1, in part L2).
//
// Measured: 16,384 rows of 5,120 with a residual 103 us, 6.5 TB/s; one row 1.75
// us, 32 rows to 8 bits 2.8 us (0.18 of it for the weight, which is read after
// the wait for the kernel before: that one may have written it).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sv_ptx.cuh"

namespace sv {

constexpr int RN_GROUP = 128;                   // columns of an 8-bit output's scale
constexpr int RN_MAX_THREADS = 1024;
constexpr int RN_ODD_MAX_D = 8 * 8 * RN_MAX_THREADS - 16;  // columns of a row that is not 16-byte aligned
constexpr float RN_FP8_MAX = 448.f;
constexpr float RN_MIN_SCALE = 1.17549435e-38f; // 2^-126: an all-zero group's scale, and the smallest

struct NormParams {
    const uint16_t *x, *residual, *weight;      // bf16 bits; residual may be null
    uint16_t *residual_out;                     // null without a residual
    uint16_t *y;                                // bf16 output, or
    uint8_t *y8;                                // e4m3 output
    float *scales;                              // e4m3: [T][lds]
    long long ldx, ldr, ldro, ldy, lds;         // elements from row to row
    int D;
    float eps, w_add;                           // w_add: 1 when the weight is stored as an offset from 1
    int row_scale;                              // e4m3: one scale per row
};

// max that keeps a NaN: a group holding one gets a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// VEC columns as they are stored: bf16 bits, two per word (VEC = 8) or one.
template <int VEC>
struct RnPiece {
    uint32_t u[VEC == 8 ? 4 : 1];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (uint32_t &w : u) w = 0u;
    }
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        if constexpr (VEC == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            u[0] = v.x;
            u[1] = v.y;
            u[2] = v.z;
            u[3] = v.w;
        } else {
            u[0] = *p;
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const
    {
        if constexpr (VEC == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else
            *p = static_cast<uint16_t>(u[0]);
    }
    // VEC = 8: columns c .. c + 7 of a row of D at `p` with any address; those
    // outside the row are zero, and not stored
    __device__ __forceinline__ void load_any(const uint16_t *p, int c, int D)
    {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t lo = c + e >= 0 && c + e < D ? p[c + e] : 0u, hi = c + e + 1 >= 0 && c + e + 1 < D ? p[c + e + 1] : 0u;
            u[e / 2] = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ void store_any(uint16_t *p, int c, int D) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e >= 0 && c + e < D) p[c + e] = static_cast<uint16_t>((e & 1) ? u[e / 2] >> 16 : u[e / 2]);
    }
    __device__ __forceinline__ float get(int e) const
    {
        return __uint_as_float((e & 1) ? (u[e >> 1] & 0xFFFF0000u) : (u[e >> 1] << 16));
    }
    // f(column, value) -> the new values, rounded to bf16
    template <class F>
    __device__ __forceinline__ void map(F f)
    {
#pragma unroll
        for (int w = 0; w < (VEC == 8 ? 4 : 1); ++w) {
            const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(f(2 * w, get(2 * w))));
            u[w] = VEC == 8 ? lo | (static_cast<uint32_t>(__bfloat16_as_ushort(
                                        __float2bfloat16_rn(f(2 * w + 1, get(2 * w + 1)))))
                                    << 16)
                            : lo;
        }
    }
};

__device__ __forceinline__ uint32_t rn_e4m3(float a)
{
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3));
}

// Piece j of thread tid holds columns VEC * (tid + j * threads) ...  ODD: rows
// at any address, the same modulo 16 bytes in all tensors but the weight: the
// pieces are those between 16-byte boundaries, the first and the last of a row
// in part.
template <int VEC, int VPT, bool FP8, bool ODD>
__global__ void __launch_bounds__(RN_MAX_THREADS) rmsnorm_kernel(const NormParams p)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nwarp = nthr >> 5;
    const long long row = blockIdx.x;
    // pieces of a row; ODD: columns of the first before the row
    const int before = ODD ? static_cast<int>(reinterpret_cast<uintptr_t>(p.x + row * p.ldx) >> 1) & 7 : 0;
    const int n = ODD ? (p.D + before + 7) >> 3 : p.D / VEC;
    auto load = [&](RnPiece<VEC> &q, const uint16_t *r, int i) {
        const int c = i * VEC - before;
        if constexpr (ODD) {
            if (c < 0 || c + VEC > p.D) {
                q.load_any(r, c, p.D);
                return;
            }
        }
        q.load(r + c);
    };
    auto store = [&](const RnPiece<VEC> &q, uint16_t *r, int i) {
        const int c = i * VEC - before;
        if constexpr (ODD) {
            if (c < 0 || c + VEC > p.D) {
                q.store_any(r, c, p.D);
                return;
            }
        }
        q.store(r + c);
    };
    auto load_weight = [&](RnPiece<VEC> &q, int i) {
        if constexpr (ODD)
            q.load_any(p.weight, i * VEC - before, p.D);
        else
            q.load(p.weight + i * VEC);
    };
    __shared__ float part[32];
    __shared__ unsigned group_max[FP8 && ODD ? RN_ODD_MAX_D / RN_GROUP + 1 : 1];    // bits of each group's largest |s w|
    pdl_launch_dependents();
    pdl_wait_prior();                           // x, and the weight too, may come from the kernel before
    // A short row's weight is read with x, a longer one's (more registers)
    // when it is used.
    constexpr bool W_KEPT = VPT <= 2;
    RnPiece<VEC> w[W_KEPT ? VPT : 1], s[VPT];
    float sum = 0.f;
    {
        const uint16_t *x = p.x + row * p.ldx;
        const uint16_t *r = p.residual ? p.residual + row * p.ldr : nullptr;
        RnPiece<VEC> b[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nthr;
            s[j].zero();
            b[j].zero();
            if (i < n) load(s[j], x, i);
            if (r && i < n) load(b[j], r, i);
        }
        if constexpr (W_KEPT)
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = tid + j * nthr;
                w[j].zero();
                if (i < n) load_weight(w[j], i);
            }
        if (r) {
            uint16_t *ro = p.residual_out + row * p.ldro;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = tid + j * nthr;
                s[j].map([&](int e, float v) { return v + b[j].get(e); });
                if (i < n) store(s[j], ro, i);
            }
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum = fmaf(s[j].get(e), s[j].get(e), sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) part[warp] = sum;
    if constexpr (FP8 && ODD)
        for (int i = tid; i <= p.D / RN_GROUP; i += nthr) group_max[i] = 0u;
    __syncthreads();
    sum = lane < nwarp ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float inv = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
    auto weight = [&](int j, int i) {
        if constexpr (W_KEPT) return w[j];
        RnPiece<VEC> v;
        load_weight(v, i);
        return v;
    };
    auto norm = [&](float v, float wv) { return v * inv * (wv + p.w_add); };

    if constexpr (!FP8) {
        uint16_t *y = p.y + row * p.ldy;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nthr;
            if (i < n) {
                const RnPiece<VEC> wj = weight(j, i);
                s[j].map([&](int e, float v) { return norm(v, wj.get(e)); });
                store(s[j], y, i);
            }
        }
    } else {
        uint8_t *y = p.y8 + row * p.ldy;
        float *sc = p.scales + row * p.lds;
        float m[VPT];                           // largest |s w| of the piece's group
        float rowmax = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nthr;
            m[j] = 0.f;
            if (i < n) {
                const RnPiece<VEC> wj = weight(j, i);
#pragma unroll
                for (int e = 0; e < VEC; ++e) m[j] = max_nan(m[j], fabsf(s[j].get(e) * (wj.get(e) + p.w_add)));
            }
            rowmax = max_nan(rowmax, m[j]);
        }
        // the largest over `width` lanes of a warp, a power of two
        auto lanes_max = [](float v, int width) {
            for (int o = width / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            return v;
        };
        if (p.row_scale) {
            rowmax = lanes_max(rowmax, 32);
            __syncthreads();                    // the sums in `part` have been read
            if (lane == 0) part[warp] = rowmax;
            __syncthreads();
            rowmax = lanes_max(lane < nwarp ? part[lane] : 0.f, 32);
#pragma unroll
            for (int j = 0; j < VPT; ++j) m[j] = rowmax;
        } else if (ODD) {                       // pieces straddle groups
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = tid + j * nthr, c = i * VEC - before;
                if (i >= n) continue;
                const RnPiece<VEC> wj = weight(j, i);
                const int g0 = max(c, 0) / RN_GROUP, end = (g0 + 1) * RN_GROUP;
                float a = 0.f, b = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float z = fabsf(s[j].get(e) * (wj.get(e) + p.w_add));
                    if (c + e < end)
                        a = max_nan(a, z);
                    else
                        b = max_nan(b, z);
                }
                // (non-negative floats compare as their bits, a NaN above all)
                atomicMax(&group_max[g0], __float_as_uint(a));
                if (c + VEC > end && end < p.D) atomicMax(&group_max[g0 + 1], __float_as_uint(b));
            }
            __syncthreads();
        } else if (VEC == 8) {                  // a group is a half warp's pieces
#pragma unroll
            for (int j = 0; j < VPT; ++j) m[j] = lanes_max(m[j], RN_GROUP / 8);
        } else {                                // a group is four warps' columns
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const float wm = lanes_max(m[j], 32);
                __syncthreads();
                if (lane == 0) part[warp] = wm;
                __syncthreads();
                const int w0 = warp & ~3;
                m[j] = max_nan(max_nan(part[w0], part[w0 + 1]), max_nan(part[w0 + 2], part[w0 + 3]));
            }
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nthr;
            auto scale_of = [&](float most) { return max_nan(most * inv / RN_FP8_MAX, RN_MIN_SCALE); };
            if (i < n) {
                const int col = i * VEC - before;
                const RnPiece<VEC> wj = weight(j, i);
                // ODD: the group of the piece's first columns and the next one
                const int g0 = max(col, 0) / RN_GROUP, end = (g0 + 1) * RN_GROUP;
                const bool grouped = ODD && !p.row_scale, two = grouped && col + VEC > end && end < p.D;
                const float m0 = grouped ? __uint_as_float(group_max[ODD ? g0 : 0]) : m[j], scale0 = scale_of(m0);
                const float m1 = two ? __uint_as_float(group_max[ODD ? g0 + 1 : 0]) : m0, scale1 = two ? scale_of(m1) : scale0;
                // at the smallest scale (and for NaNs) the quotient itself
                auto quant = [&](int e) {
                    const float z = s[j].get(e) * (wj.get(e) + p.w_add);
                    const bool second = two && col + e >= end;
                    const float scale = second ? scale1 : scale0, most = second ? m1 : m0;
                    return rn_e4m3(scale > RN_MIN_SCALE ? z * RN_FP8_MAX / most : z * inv / scale);
                };
                if (p.row_scale) {
                    if (col <= 0) sc[0] = scale0;
                } else {
                    if (col <= g0 * RN_GROUP) sc[g0] = scale0;
                    if (two) sc[g0 + 1] = scale1;
                }
                if constexpr (VEC == 8) {
                    uint32_t lo = 0u, hi = 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        lo |= quant(e) << (8 * e);
                        hi |= quant(e + 4) << (8 * e);
                    }
                    if (ODD && (col < 0 || col + VEC > p.D)) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (col + e >= 0 && col + e < p.D) y[col + e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
                    } else {
                        *reinterpret_cast<uint2 *>(y + col) = make_uint2(lo, hi);
                    }
                } else {
                    y[col] = static_cast<uint8_t>(quant(0));
                }
            }
        }
    }
}

}  // namespace sv
