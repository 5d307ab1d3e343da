// w4a16_gate_up.cuh -- the first half of a gated feed-forward block from int4
// weights: h = act(x Wg^T) * (x Wu^T), both projections, the activation and
// the product in one pass over the packed weights.
// w4a16_gate_up_tc.cuh has the form for wide projections; this one is the
// quicker for narrow ones and few tokens, where its time goes with the weights.
//
// Wq holds the F gate rows and then the F up rows in the library's W4A16
// format.  The m16n8k16 MMA leaves rows g and g + 8 of its A operand in the
// same thread, so a tile is eight gate rows (A rows 0..7) and the same eight
// up rows (A rows 8..15): a thread ends with the gate and the up value of
// its column and tokens, and the product needs no exchange.
//
// A warp owns a tile and walks K; its packed words go through its own ring in
// shared memory by 16-byte cp.async (a lane reads back only what it copied,
// so the ring needs no barrier), deep enough to keep HBM busy: GU_STAGES
// groups of 1 KB a warp.  With fewer than 16 tiles a block, KS = 2..16 warps
// share a tile's groups and add their sums in shared memory in a fixed
// order.  The activations are shared by the block: chunks of K, bf16, in
// B-fragment order, double-buffered.
//
// Group scales multiply each group's fp32 sum, as in w4a16_gemm; levels and
// activations are exact in bf16 and their products in fp32.  The gate and up
// sums are not rounded before the activation and the product.
#pragma once

#include "sv_ptx.cuh"
#include "w4a16_stream.cuh"

namespace sv {

constexpr int GU_WARPS = 16;
constexpr int GU_STAGES = 8;                    // groups of a warp's ring
constexpr int GU_UNIT = 1024;                   // bytes of a tile's group: 16 rows x 64
constexpr int GU_ROW_PAD = 16;                  // bytes after a token's chunk: B loads free of bank conflicts
constexpr int GU_MAX_TOKENS = 32;

enum { GU_SILU = 0, GU_GELU_TANH = 1 };

// Groups of an activation chunk: 16 with one token tile, 8 with two, 4 with four.
__host__ __device__ constexpr int gu_chunk_groups(int NT) { return 16 / NT; }
__host__ __device__ constexpr int gu_row_bytes(int NT) { return gu_chunk_groups(NT) * 256 + GU_ROW_PAD; }
__host__ __device__ constexpr int gu_chunk_bytes(int NT) { return 8 * NT * gu_row_bytes(NT); }
__host__ __device__ constexpr int gu_smem_bytes(int NT) { return GU_WARPS * GU_STAGES * GU_UNIT + 2 * gu_chunk_bytes(NT); }

struct GateUpParams {
    const uint16_t *x;                          // [T][K] bf16 bits
    const uint32_t *Wq;                         // [2F][K/8]
    const uint16_t *scales;                     // [2F][K/128]
    uint16_t *h;                                // [T][F]
    int T, K, G, F;
    int tiles;                                  // ceil(F / 8)
    int ks_log;                                 // log2 of the warps that share a tile
    int act;
};

// silu: g / (1 + e^-g); gelu in its tanh form: g (1 + tanh z) / 2 = g / (1 +
// e^-2z), which loses nothing where tanh z is near -1 (g < -5: 0 or 30 % off).
__device__ __forceinline__ float gu_act(float g, int act)
{
    const float z = act == GU_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g / (1.f + __expf(-z));
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int NT>
__global__ void __launch_bounds__(GU_WARPS * 32, 1) w4a16_gate_up_kernel(const GateUpParams p)
{
    extern __shared__ __align__(128) uint8_t gu_smem[];
    constexpr int CG = gu_chunk_groups(NT), ROWB = gu_row_bytes(NT), CHUNKB = gu_chunk_bytes(NT);
    constexpr int PIECES = 8 * NT * CG * 16;    // 16-byte pieces of a chunk: 2048
    constexpr int PPT = PIECES / (GU_WARPS * 32);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_addr(gu_smem) + static_cast<uint32_t>(warp * GU_STAGES * GU_UNIT + lane * 16);
    uint8_t *xs = gu_smem + GU_WARPS * GU_STAGES * GU_UNIT;
    const int ks = 1 << p.ks_log, slots = GU_WARPS >> p.ks_log;
    const int kpart = warp & (ks - 1), tslot = warp >> p.ks_log;
    const int G = p.G, n_chunk = (G + CG - 1) / CG;
    const int t_first = static_cast<int>(static_cast<long long>(blockIdx.x) * p.tiles / gridDim.x);
    const int t_last = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * p.tiles / gridDim.x);
    const uint64_t pol = policy_evict_first();
    const uint32_t xsw = static_cast<uint32_t>((c & 2) * 16);
    bool waited = false;
    pdl_launch_dependents();

    for (int tb = t_first; tb < t_last; tb += slots) {
        const int tile = tb + tslot;
        const bool on = tile < t_last;
        // this lane's rows: column 8 tile + g of the gate and of the up half
        // (columns past F read the last row and are not stored)
        const int col = min((on ? tile : t_first) * 8 + g, p.F - 1);
        const size_t rg = static_cast<size_t>(col), ru = rg + static_cast<size_t>(p.F);
        const uint8_t *wg = reinterpret_cast<const uint8_t *>(p.Wq) + rg * (static_cast<size_t>(p.K) / 2) + c * 16;
        const uint8_t *wu = reinterpret_cast<const uint8_t *>(p.Wq) + ru * (static_cast<size_t>(p.K) / 2) + c * 16;
        const uint16_t *sg = p.scales + rg * G, *su = p.scales + ru * G;
        const int mine = on ? (G - kpart + ks - 1) >> p.ks_log : 0;     // groups kpart, kpart + ks, ...
        auto issue = [&](int i) {
            if (i < mine) {
                const uint32_t dst = ring + static_cast<uint32_t>((i & (GU_STAGES - 1)) * GU_UNIT);
                const size_t off = static_cast<size_t>(kpart + (i << p.ks_log)) * 64;
                cp_async_16_hint(dst, wg + off, pol);
                cp_async_16_hint(dst + 512, wu + off, pol);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < GU_STAGES - 1; ++i) issue(i);
        if (!waited) {
            pdl_wait_prior();                   // activations may come from the previous kernel
            waited = true;
        }
        // one chunk of activations: global -> registers, -> shared memory in
        // B-fragment order (x0,x4)(x1,x5)(x2,x6)(x3,x7), as the nibbles pair
        uint4 xr[PPT];
        auto x_load = [&](int ch) {
#pragma unroll
            for (int u = 0; u < PPT; ++u) {
                const int i = threadIdx.x + u * GU_WARPS * 32, t = i / (CG * 16), j = ch * CG * 16 + i % (CG * 16);
                xr[u] = (t < p.T && j < G * 16)
                            ? __ldg(reinterpret_cast<const uint4 *>(p.x) + static_cast<size_t>(t) * (p.K / 8) + j)
                            : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto x_store = [&](int ch) {
            uint8_t *buf = xs + (ch & 1) * CHUNKB;
#pragma unroll
            for (int u = 0; u < PPT; ++u) {
                const int i = threadIdx.x + u * GU_WARPS * 32, t = i / (CG * 16), j = i % (CG * 16);
                const uint4 v = xr[u];
                *reinterpret_cast<uint4 *>(buf + t * ROWB + ((j & ~15) + chunk_slot(j & 15)) * 16) =
                    make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                               __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
            }
        };
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
        x_load(0);
        x_store(0);
        __syncthreads();
        int i = 0;
        // scales of the warp's next group, read one group ahead
        uint32_t s_g = mine > 0 ? ldg_u16(sg + kpart) : 0u, s_u = mine > 0 ? ldg_u16(su + kpart) : 0u;
        for (int ch = 0; ch < n_chunk; ++ch) {
            if (ch + 1 < n_chunk) x_load(ch + 1);
            const uint32_t xb = smem_addr(xs + (ch & 1) * CHUNKB) + static_cast<uint32_t>(g * ROWB + c * 64);
            const int g_end = min(G, (ch + 1) * CG);
            for (; i < mine; ++i) {
                const int grp = kpart + (i << p.ks_log);
                if (grp >= g_end) break;
                cp_async_wait<GU_STAGES - 2>();
                const uint32_t wa_addr = ring + static_cast<uint32_t>((i & (GU_STAGES - 1)) * GU_UNIT);
                const uint4 wa = lds128(wa_addr), wb = lds128(wa_addr + 512);
                issue(i + GU_STAGES - 1);
                const float f_g = bf16_bits_to_float(s_g), f_u = bf16_bits_to_float(s_u);
                if (i + 1 < mine) {
                    s_g = ldg_u16(sg + grp + ks);
                    s_u = ldg_u16(su + grp + ks);
                }
                const uint32_t xg = xb + static_cast<uint32_t>((grp - ch * CG) * 256);
                float ga[NT][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t wA = (m == 0) ? wa.x : (m == 1) ? wa.y : (m == 2) ? wa.z : wa.w;
                    const uint32_t wB = (m == 0) ? wb.x : (m == 1) ? wb.y : (m == 2) ? wb.z : wb.w;
                    uint32_t a[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        a[2 * q] = dequant2(wA >> (4 * q));
                        a[2 * q + 1] = dequant2(wB >> (4 * q));
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 v = lds128(xg + static_cast<uint32_t>(nt * 8 * ROWB) + ((16u * m) ^ xsw));
                        if (m == 0)
                            mma_bf16_16816_zc(ga[nt], a[0], a[1], a[2], a[3], v.x, v.y);
                        else
                            mma_bf16_16816(ga[nt], a[0], a[1], a[2], a[3], v.x, v.y);
                        mma_bf16_16816(ga[nt], a[4], a[5], a[6], a[7], v.z, v.w);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    acc[nt][0] = fmaf(f_g, ga[nt][0], acc[nt][0]);
                    acc[nt][1] = fmaf(f_g, ga[nt][1], acc[nt][1]);
                    acc[nt][2] = fmaf(f_u, ga[nt][2], acc[nt][2]);
                    acc[nt][3] = fmaf(f_u, ga[nt][3], acc[nt][3]);
                }
            }
            if (ch + 1 < n_chunk) x_store(ch + 1);
            __syncthreads();
        }
        cp_async_wait<0>();                     // (empty groups only)
        if (ks > 1) {
            // the parts of a tile, added in order by its first warp; every
            // warp is past its last read of the activations
            float *red = reinterpret_cast<float *>(xs) + (warp * 32 + lane) * 4 * NT;
            if (kpart > 0)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    *reinterpret_cast<float4 *>(red + 4 * nt) = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
            __syncthreads();
            if (kpart == 0)
                for (int j = 1; j < ks; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 v = *reinterpret_cast<const float4 *>(red + j * 32 * 4 * NT + 4 * nt);
                        acc[nt][0] += v.x;
                        acc[nt][1] += v.y;
                        acc[nt][2] += v.z;
                        acc[nt][3] += v.w;
                    }
        }
        const int out = tile * 8 + g;
        if (on && kpart == 0 && out < p.F)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = nt * 8 + 2 * c + e;
                    if (t < p.T)
                        p.h[static_cast<size_t>(t) * p.F + out] =
                            __bfloat16_as_ushort(__float2bfloat16_rn(gu_act(acc[nt][e], p.act) * acc[nt][2 + e]));
                }
        __syncthreads();                        // the activation buffers are free again
    }
}

}  // namespace sv
