// tc_ops.cuh -- tensor-memory stores of several widths, descriptors of
// 128-byte swizzled operands and the two-term bf16 split, for the layer
// operators' tcgen05 kernels.
#pragma once

#include <cstdint>

#include "gated_delta.cuh"
#include "sv_ptx.cuh"
#include "w4a16_stream.cuh"

namespace sv {

// Two floats -> bf16x2 (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// a and b as two bf16 terms each: hi the value rounded, lo what is left
// rounded; together 16 bits of each.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(a, b);
    lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}

// Two fp32 values as tensor memory gives them, as a packed pair.
__device__ __forceinline__ f32x2 pair_x2(uint32_t lo, uint32_t hi)
{
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}

// The split of a packed pair.
__device__ __forceinline__ void split_bf16x2(f32x2 v, uint32_t &hi, uint32_t &lo)
{
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    hi = pack_bf16x2(__uint_as_float(a), __uint_as_float(b));
    f32x2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(v), "l"(pair_x2(hi << 16, hi & 0xFFFF0000u)));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(r));
    lo = pack_bf16x2(__uint_as_float(a), __uint_as_float(b));
}

// Shared-memory descriptor of an operand whose rows run along the products'
// K: 64 columns (128 bytes) a row, 16-byte pieces swizzled within eight rows
// (layout 2 at bits 61-63), 1024 bytes from one eight rows to the next
// (stride byte offset >> 4 at bits 32-45), descriptor version 1 (bits 46-48).
// A step of 16 columns along K is 32 bytes further.
__device__ __forceinline__ uint64_t desc_k_sw128(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// The same tile read across: its rows are the products' K and its 64
// columns their N.  Eight rows along K are 1024 bytes, the next 64 columns
// along N 8192 bytes (leading byte offset >> 4 at bits 16-29) further; a step
// of 16 rows along K is 2048 bytes, one of 16 columns along N 32 bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// This thread's N registers -> N consecutive tensor-memory columns of its lane.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[N])
{
    static_assert(N == 8 || N == 16, "widths in use");
    if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
                     "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                     ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                       "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
                       "r"(v[15])
                     : "memory");
}

// N consecutive tensor-memory columns of this thread's lane -> N registers.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N])
{
    static_assert(N == 16, "the width in use");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(taddr)
                 : "memory");
}

// Whether the phase of that parity has completed; the thread may sleep up to
// `ns` nanoseconds for it, so that waiting warps take no issue slots.
__device__ __forceinline__ bool mbar_sleep_wait(uint32_t bar, uint32_t parity, uint32_t ns)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(ns) : "memory");
    return ok != 0;
}

// Start a later copy's way from HBM: the bytes (a multiple of 16, 16-byte
// aligned), or a box of a tensor map, into L2.
__device__ __forceinline__ void prefetch_l2(const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void prefetch_l2_2d(const void *tmap, int c0, int c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1) : "memory");
}

// Instruction descriptor of an M = 128 product of N = n columns: bf16
// operands, fp32 accumulator; B's rows along the products' K, or across.
constexpr uint32_t tc_idesc_bf16(int n, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// The rare long wait, out of line: the roles' loops share the instruction cache.
static __device__ __noinline__ void tc_long_wait(uint32_t bar, uint32_t parity, volatile int *flag, int *err)
{
    if (mbar_wait_bounded(bar, parity, *flag ? WAIT_LIMIT_AFTER_ERR_NS : WAIT_LIMIT_NS)) return;
    *flag = 1;
    atomicOr(err, 2);
}

// Whole warps wait (with one lane polling for the others the gated delta
// scan took 298 instead of 255 us).
struct TcWait {
    volatile int *flag;                         // in shared memory: a wait ran out
    int *err;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const
    {
        if (!mbar_sleep_wait(bar, parity & 1u, 100000u)) tc_long_wait(bar, parity & 1u, flag, err);
    }
};

}  // namespace sv
