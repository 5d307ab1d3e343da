// layer_ops.cu -- the C ABI of what a hybrid decoder layer runs between its
// weight reads (include/specverify.h): argument checks, launch shapes and
// dispatch of the norm, gated delta rule and gated feed-forward kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "gated_delta.cuh"
#include "gated_delta_chunk.cuh"
#include "rmsnorm.cuh"
#include "specverify.h"
#include "sv_host.h"
#include "w4a16_gate_up.cuh"
#include "w4a16_gate_up_tc.cuh"

namespace sv {
namespace {

constexpr int MAX_DEVICES = 64;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Tensor map of `rows` rows of `cols` values, `pitch` bytes apart; boxes of
// `height` rows and `width` values, 128-byte swizzled where asked.
int encode_rows(CUtensorMap *m, CUtensorMapDataType type, const void *base, long long cols, long long rows,
                long long pitch, int width, int height, bool swizzled)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(height)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = g_encode(m, type, 2, const_cast<void *>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE,
                                swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SV_OK : SV_ERR_CUDA;
}

// bf16 rows, `ld` values apart, in boxes of a block of prompt rows.
int encode_blocks(CUtensorMap *m, const void *base, long long cols, long long rows, long long ld, int width, bool swizzled)
{
    return encode_rows(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, cols, rows, 2 * ld, width, DC_ROWS, swizzled);
}

template <class F>
cudaError_t raise(F *kernel, int bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DK>
cudaError_t delta_block_raise();

// The current device's facts, with the kernels' shared-memory limits raised
// once per device.
int ops_device(DeviceInfo *out)
{
    const int rc = device_info(out);
    if (rc != SV_OK) return rc;
    static std::mutex mu;
    static bool ready[MAX_DEVICES] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (ready[out->dev]) return SV_OK;
    cudaError_t e = cudaSuccess;
    auto up = [&](cudaError_t r) { e = e != cudaSuccess ? e : r; };
    up(delta_block_raise<64>());
    up(delta_block_raise<128>());
    up(raise(delta_prep_kernel<64>, sizeof(DcPrepSmem<64>)));
    up(raise(delta_prep_kernel<128>, sizeof(DcPrepSmem<128>)));
    up(raise(delta_scan_kernel<64>, DsSmem<64>::BYTES));
    up(raise(delta_scan_kernel<128>, DsSmem<128>::BYTES));
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        up(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q));
        if (e == cudaSuccess && (q != cudaDriverEntryPointSuccess || !fn)) return SV_ERR_CUDA;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    up(raise(w4a16_gate_up_kernel<1>, gu_smem_bytes(1)));
    up(raise(w4a16_gate_up_kernel<2>, gu_smem_bytes(2)));
    up(raise(w4a16_gate_up_kernel<4>, gu_smem_bytes(4)));
    up(raise(w4a16_gate_up_tc_kernel<16>, GtSmem<16>::BYTES));
    up(raise(w4a16_gate_up_tc_kernel<32>, GtSmem<32>::BYTES));
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

// ----------------------------------------------------------------- norm

constexpr int NORM_MAX_D = 65536;

int check_norm(const sv_bf16 *x, long long ldx, const sv_bf16 *residual, long long ldr, const sv_bf16 *weight, int T,
               int D, float eps, int flags, const sv_bf16 *residual_out, long long ldro, const void *y, long long ldy)
{
    if (T < 0 || D < 1 || D > NORM_MAX_D) return SV_ERR_SHAPE;
    if (!(eps >= 0.f) || (flags & ~SV_NORM_UNIT_OFFSET)) return SV_ERR_SHAPE;
    if (ldx < D || ldy < D || (residual && (ldr < D || ldro < D))) return SV_ERR_SHAPE;
    if (T == 0) return SV_OK;                    // (tensors without rows have no addresses)
    if (!x || !weight || !y || (residual && !residual_out) || (!residual && residual_out)) return SV_ERR_NULL;
    if (!aligned_to(x, 2) || !aligned_to(weight, 2) || !aligned_to(residual, 2) || !aligned_to(residual_out, 2))
        return SV_ERR_ALIGN;
    return SV_OK;
}

template <int VEC, bool FP8, bool ODD = false>
int norm_launch(const NormParams &p, int T, int vpt, int threads, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(T));
    switch (vpt) {
    case 1: return launch(rmsnorm_kernel<VEC, 1, FP8, ODD>, grid, threads, 0, stream, p);
    case 2: return launch(rmsnorm_kernel<VEC, 2, FP8, ODD>, grid, threads, 0, stream, p);
    case 4: return launch(rmsnorm_kernel<VEC, 4, FP8, ODD>, grid, threads, 0, stream, p);
    case 8: return launch(rmsnorm_kernel<VEC, 8, FP8, ODD>, grid, threads, 0, stream, p);
    default: break;
    }
    if constexpr (VEC == 1) {
        if (vpt == 16) return launch(rmsnorm_kernel<VEC, 16, FP8, ODD>, grid, threads, 0, stream, p);
        return launch(rmsnorm_kernel<VEC, 64, FP8, ODD>, grid, threads, 0, stream, p);
    }
    return SV_ERR_SHAPE;
}

template <bool FP8>
int norm_call(NormParams p, int T, cudaStream_t stream)
{
    if (T == 0) return SV_OK;
    DeviceInfo dev;
    const int rc = ops_device(&dev);
    if (rc != SV_OK) return rc;
    const bool wide = p.D % 8 == 0 && p.ldx % 8 == 0 && p.ldy % 8 == 0 && aligned_to(p.x, 16) &&
                      aligned_to(p.weight, 16) && aligned_to(FP8 ? static_cast<const void *>(p.y8) : p.y, FP8 ? 8 : 16) &&
                      (!p.residual || (p.ldr % 8 == 0 && p.ldro % 8 == 0 && aligned_to(p.residual, 16) &&
                                       aligned_to(p.residual_out, 16)));
    // rows that are not 16-byte aligned, but all off by as much (odd lengths):
    // 16-byte pieces all the same.  16,384 rows of 1,001 / 5,119 columns 28 /
    // 167 us (one column a thread 87 / 666), of 5,119 to 8 bits 454 (909), one
    // row of 5,119 2.0 (4.6); a few short rows are quicker by columns (one of
    // 1,001 1.4, by pieces 1.7)
    auto off = [](const void *a, long long ld, int log) { return ((reinterpret_cast<uintptr_t>(a) >> log) & 7) * 8 + (ld & 7); };
    const unsigned long long at = off(p.x, p.ldx, 1);
    const bool odd = !wide && p.D >= 64 && 1LL * T * p.D >= 2048 && p.D <= RN_ODD_MAX_D &&
                     (FP8 ? off(p.y8, p.ldy, 0) : off(p.y, p.ldy, 1)) == at &&
                     (!p.residual || (off(p.residual, p.ldr, 1) == at && off(p.residual_out, p.ldro, 1) == at));
    const int n = wide ? p.D / 8 : odd ? p.D / 8 + 2 : p.D;     // most pieces of a row
    int vpt = 1;
    while (n > vpt * RN_MAX_THREADS) vpt *= 2;
    if (!wide && vpt == 32) vpt = 64;
    const int per = 128;                         // the scalar 8-bit path groups four warps
    const int threads = ((n + vpt - 1) / vpt + per - 1) / per * per;
    if (odd) return norm_launch<8, FP8, true>(p, T, vpt, threads, stream);
    return wide ? norm_launch<8, FP8>(p, T, vpt, threads, stream) : norm_launch<1, FP8>(p, T, vpt, threads, stream);
}

// ----------------------------------------------------- gated delta rule

int check_delta_shape(const sv_delta_shape *s)
{
    if (!s) return SV_ERR_NULL;
    if (s->Hk < 1 || s->Hv < 1 || s->Hv > 65535 || s->Hv % s->Hk) return SV_ERR_SHAPE;
    if ((s->dk != 64 && s->dk != 128) || (s->dv != 64 && s->dv != 128)) return SV_ERR_SHAPE;
    if (s->scale != s->scale || (s->flags & ~(SV_DELTA_L2NORM | SV_DELTA_COMMIT | SV_DELTA_ZERO_INIT))) return SV_ERR_SHAPE;
    return SV_OK;
}

int check_delta_rows(const sv_delta_rows *r, const sv_delta_shape *s, bool want_q)
{
    if (!r) return SV_ERR_NULL;
    if ((want_q && !r->q) || !r->k || !r->v || !r->g || !r->beta) return SV_ERR_NULL;
    const long long nk = static_cast<long long>(s->Hk) * s->dk, nv = static_cast<long long>(s->Hv) * s->dv;
    if ((want_q && r->ldq < nk) || r->ldk < nk || r->ldv < nv || r->ldg < s->Hv) return SV_ERR_SHAPE;
    if ((want_q && (r->ldq % 8 || !aligned_to(r->q, 16))) || r->ldk % 8 || r->ldv % 8 || !aligned_to(r->k, 16) ||
        !aligned_to(r->v, 16) || !aligned_to(r->g, 4) || !aligned_to(r->beta, 4))
        return SV_ERR_ALIGN;
    return SV_OK;
}

int check_delta_state(const sv_delta_shape *s, const float *state, const int32_t *state_idx, int n_slots, int B)
{
    if (B < 0 || B > 65535 || n_slots < 1 || (!state_idx && n_slots < B)) return SV_ERR_SHAPE;
    if (!state) return SV_ERR_NULL;
    if (!aligned_to(state, 16) || !aligned_to(state_idx, 4)) return SV_ERR_ALIGN;
    return SV_OK;
}

int check_delta_out(const sv_delta_shape *s, const sv_bf16 *o, long long ldo)
{
    if (!o) return SV_ERR_NULL;
    if (ldo < static_cast<long long>(s->Hv) * s->dv) return SV_ERR_SHAPE;
    if (ldo % 8 || !aligned_to(o, 16)) return SV_ERR_ALIGN;
    return SV_OK;
}

DeltaRows delta_rows(const sv_delta_rows *r)
{
    if (!r) return DeltaRows{};
    return DeltaRows{r->q, r->k, r->v, r->g, r->beta, r->ldq, r->ldk, r->ldv, r->ldg};
}

DeltaParams delta_params(const sv_delta_rows *rows, const sv_delta_shape *s, float *state, const int32_t *state_idx,
                         int n_slots, sv_bf16 *o, long long ldo, const DeviceInfo &dev)
{
    DeltaParams p{};
    p.rows = delta_rows(rows);
    p.Hk = s->Hk;
    p.Hv = s->Hv;
    p.dv = s->dv;
    p.scale = s->scale;
    p.l2norm = (s->flags & SV_DELTA_L2NORM) != 0;
    p.commit = (s->flags & SV_DELTA_COMMIT) != 0;
    p.state = state;
    p.state_idx = state_idx;
    p.n_slots = n_slots;
    p.o = o;
    p.ldo = ldo;
    p.err = dev.err;
    return p;
}

// Whether a step runs row by row (gated_delta_step_kernel) or takes its rows
// all at once (gated_delta_block_kernel).  One or two rows whose state is a
// wave of small blocks at most are quicker without the second kernel's tiles:
// 48 heads of 128 x 128, one row, 1 / 4 sequences 3.8 / 6.0 us against 5.4 /
// 9.0, two rows 4.1 / 6.9 against 5.5 / 9.2.  Beyond that its asynchronous
// copies win: 16 / 64 / 256 sequences of two rows 19 / 66 / 244 us against
// 21 / 100 / 389, and so do its tiles with more rows: 4 and 4 rows of 1 / 4
// sequences 5.8 / 9.6 us, row by row 7.0 / 11.7.
bool delta_step_by_rows(int rows, long long state_rows, const DeviceInfo &dev)
{
    return rows < 3 && state_rows <= 5LL * GB_COLS * dev.sms;
}

// Whether a block of up to 16 rows has two warps for 16 state rows.  With two
// or three blocks a multiprocessor the chain of a block counts, which that
// shortens, whatever the rows: 48 heads of 128 x 128, 4 and 4 rows (all, one or
// none replayed) of 2 sequences 7.3 / 7.0 / 5.0 us against 8.7 / 8.3 / 5.4, of 4
// 7.6 / 7.3 / 5.1 against 9.9 / 9.6 / 6.3; 8 and 8 of 2 / 4 8.9 / 9.9 against
// 10.2 / 10.7; 4 rows alone 7.0 / 7.2 against 8.4 / 9.5.  A single block (one
// sequence: 5.7 against 5.4 us) and more of them (5 sequences, 8 and 8 rows 11.6
// against 10.6; 16 of them 29 against 25) do better without.
bool delta_step_split(long long state_rows, const DeviceInfo &dev)
{
    const long long blocks = state_rows / GB_COLS;
    return blocks > dev.sms && blocks <= 3LL * dev.sms;
}

template <int DK, int NK, int NQ, int KS>
constexpr size_t delta_block_smem()
{
    return sizeof(GbSmem<DK, 8 * NK, 8 * NQ, KS>);
}

template <int DK, int NK, int NQ, int KS>
int delta_block_launch(const DeltaParams &p, int B, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(p.dv / GB_COLS), static_cast<unsigned>(p.Hv), static_cast<unsigned>(B));
    return launch(gated_delta_block_kernel<DK, NK, NQ, KS>, grid, gb_threads(KS), delta_block_smem<DK, NK, NQ, KS>(), stream, p);
}

// `split`: two warps for 16 state rows, half the columns each (up to 16 rows).
template <int DK>
int delta_block_dispatch(const DeltaParams &p, int B, bool split, cudaStream_t stream)
{
    const int nk = (p.prev_T + p.T + 7) / 8;
    if (nk <= 1) return split ? delta_block_launch<DK, 1, 1, 2>(p, B, stream) : delta_block_launch<DK, 1, 1, 1>(p, B, stream);
    if (nk <= 2 && p.T <= 8)
        return split ? delta_block_launch<DK, 2, 1, 2>(p, B, stream) : delta_block_launch<DK, 2, 1, 1>(p, B, stream);
    if (nk <= 4 && p.T <= 16) return delta_block_launch<DK, 4, 2, 1>(p, B, stream);
    return delta_block_launch<DK, 8, 4, 1>(p, B, stream);
}

template <int DK>
cudaError_t delta_block_raise()
{
    cudaError_t e = cudaSuccess;
    auto up = [&](cudaError_t r) { e = e != cudaSuccess ? e : r; };
    up(raise(gated_delta_block_kernel<DK, 1, 1, 1>, delta_block_smem<DK, 1, 1, 1>()));
    up(raise(gated_delta_block_kernel<DK, 1, 1, 2>, delta_block_smem<DK, 1, 1, 2>()));
    up(raise(gated_delta_block_kernel<DK, 2, 1, 1>, delta_block_smem<DK, 2, 1, 1>()));
    up(raise(gated_delta_block_kernel<DK, 2, 1, 2>, delta_block_smem<DK, 2, 1, 2>()));
    up(raise(gated_delta_block_kernel<DK, 4, 2, 1>, delta_block_smem<DK, 4, 2, 1>()));
    up(raise(gated_delta_block_kernel<DK, 8, 4, 1>, delta_block_smem<DK, 8, 4, 1>()));
    return e;
}

// Blocks of the workspace: every sequence's whole and part blocks.
long long delta_blocks(int R, int B) { return static_cast<long long>(R / DC_ROWS) + B; }

size_t delta_block_bytes(int R, int B, int Hv) { return static_cast<size_t>(delta_blocks(R, B)) * static_cast<size_t>(Hv) * DC_BLOCK; }

// A few rows go row by row, without blocks.  48 heads of 128 x 128, row by row
// against by blocks: one sequence of 16 / 32 / 48 / 64 rows 14 / 25 / 36 / 47 us
// against 25 / 25 / 25 / 26, four of 16 / 32 rows 24 / 43 against 39 / 39, 64 of
// 16 rows 284 against 268.  How the rows are shared out is known on the device
// only, so the limit on their number also bounds the loss where one sequence
// has them all.
bool delta_by_rows(int R, int B) { return R <= DC_ROWS && R < 32LL * B; }

template <int DK>
int delta_chunk_launch(const DeltaChunkParams &p, const DeviceInfo &dev, cudaStream_t stream)
{
    CUtensorMap tmK, tmQ, tmV;
    const DeltaRows &r = p.d.rows;
    const long long nk = static_cast<long long>(p.d.Hk) * DK, nv = static_cast<long long>(p.d.Hv) * p.d.dv;
    int rc = encode_blocks(&tmK, r.k, nk, p.R, r.ldk, 64, true);
    if (rc == SV_OK) rc = encode_blocks(&tmQ, r.q, nk, p.R, r.ldq, 64, true);
    if (rc == SV_OK) rc = encode_blocks(&tmV, r.v, nv, p.R, r.ldv, p.d.dv, false);
    if (rc != SV_OK) return rc;
    const long long blocks = delta_blocks(p.R, p.B), parts = std::min<long long>(dev.sms, blocks * p.d.Hv);
    rc = launch(delta_prep_kernel<DK>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(p.d.Hk)), 128,
                sizeof(DcPrepSmem<DK>), stream, p);
    if (rc != SV_OK) return rc;
    DeltaChunkParams s = p;
    s.cu = p.cu_run;
    return launch(delta_scan_kernel<DK>, dim3(static_cast<unsigned>(std::min<long long>(parts, DC_FLAGS / 4))), DS_THREADS,
                  DsSmem<DK>::BYTES, stream, s, tmK, tmQ, tmV);
}

// ------------------------------------------------------ gated feed-forward

// Columns of a tile of the wide kernel: the result divided evenly over the
// multiprocessors, in as few rounds of 128 lanes as hold it.
int gate_up_cols(int F, int sms)
{
    const long long rounds = (F + 1LL * sms * GT_ROWS - 1) / (1LL * sms * GT_ROWS);
    return static_cast<int>((F + sms * rounds - 1) / (sms * rounds));
}

// Whether the wide kernel (w4a16_gate_up_tc_kernel) is the quicker one.  Its
// time goes with the groups of K and the rounds (4 + 0.44 us a group up to 16
// tokens, 5 + 0.53 beyond), whatever the tile's columns, the other kernel's
// with the weights.  Measured, wide against other, K 5,120: F 9,728 (64
// columns a tile) 32 tokens 25.9 / 26.4 us; F 10,944 (72) 16 tokens 21.5 /
// 23.0, 32 tokens 26.0 / 33.4; F 12,768 (84) 8 tokens 21.1 / 18.9; F 15,048
// (99) 8 tokens 21.2 / 22.8; F 17,408 (115) 1 / 8 / 16 / 32 tokens 21.5 / 21.7 /
// 22.1 / 26.6 against 23.5 / 23.9 / 30.0 / 42.3.  With K 1,280 the wide
// kernel's start weighs more: F 17,408, 8 / 16 / 32 tokens 9.0 / 9.4 / 11.7
// against 7.5 / 9.3 / 12.9 (16 tokens: no difference).
bool gate_up_wide(int T, int G, int cols)
{
    return cols >= (T > 16 ? 54 + 430 / G : T > 8 ? 60 + 430 / G : 82 + 680 / G);
}

template <int N>
int gate_up_tc_launch(const GateUpParams &q, const DeviceInfo &dev, cudaStream_t stream)
{
    GateUpTcParams p{};
    p.scales = q.scales;
    p.h = q.h;
    p.T = q.T;
    p.G = q.G;
    p.F = q.F;
    p.act = q.act;
    p.err = dev.err;
    p.cols = gate_up_cols(q.F, dev.sms);
    p.tiles = (q.F + p.cols - 1) / p.cols;
    CUtensorMap tmW, tmX;
    int rc = encode_rows(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT32, q.Wq, q.K / 8, 2LL * q.F, q.K / 2, 32, p.cols, true);
    if (rc == SV_OK) rc = encode_rows(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q.x, q.K, q.T, 2LL * q.K, 64, N, true);
    if (rc != SV_OK) return rc;
    const unsigned grid = static_cast<unsigned>(std::min(p.tiles, dev.sms));
    return launch(w4a16_gate_up_tc_kernel<N>, dim3(grid), GT_THREADS, GtSmem<N>::BYTES, stream, p, tmW, tmX);
}

template <int NT>
int gate_up_launch(const GateUpParams &p, const DeviceInfo &dev, cudaStream_t stream)
{
    const int grid = p.tiles < dev.sms ? p.tiles : dev.sms;
    return launch(w4a16_gate_up_kernel<NT>, dim3(static_cast<unsigned>(grid)), GU_WARPS * 32, gu_smem_bytes(NT), stream, p);
}

}  // namespace
}  // namespace sv

extern "C" {

int rmsnorm_residual(const sv_bf16 *x, long long ldx, const sv_bf16 *residual, long long ldr, const sv_bf16 *weight,
                     int T, int D, float eps, int flags, sv_bf16 *residual_out, long long ldro, sv_bf16 *y,
                     long long ldy, sv_stream stream)
{
    using namespace sv;
    const int rc = check_norm(x, ldx, residual, ldr, weight, T, D, eps, flags, residual_out, ldro, y, ldy);
    if (rc != SV_OK) return rc;
    if (!aligned_to(y, 2)) return SV_ERR_ALIGN;
    NormParams p{};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.residual_out = residual_out;
    p.y = y;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldro = ldro;
    p.ldy = ldy;
    p.D = D;
    p.eps = eps;
    p.w_add = (flags & SV_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    return norm_call<false>(p, T, reinterpret_cast<cudaStream_t>(stream));
}

int rmsnorm_residual_fp8(const sv_bf16 *x, long long ldx, const sv_bf16 *residual, long long ldr,
                         const sv_bf16 *weight, int T, int D, float eps, int flags, int group, sv_bf16 *residual_out,
                         long long ldro, uint8_t *y, long long ldy, float *scales, long long lds, sv_stream stream)
{
    using namespace sv;
    const int rc = check_norm(x, ldx, residual, ldr, weight, T, D, eps, flags, residual_out, ldro, y, ldy);
    if (rc != SV_OK) return rc;
    if (group != 0 && group != RN_GROUP) return SV_ERR_SHAPE;
    if (lds < (group ? (D + group - 1) / group : 1)) return SV_ERR_SHAPE;
    if (T > 0 && !scales) return SV_ERR_NULL;
    if (!aligned_to(scales, 4)) return SV_ERR_ALIGN;
    NormParams p{};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.residual_out = residual_out;
    p.y8 = y;
    p.scales = scales;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldro = ldro;
    p.ldy = ldy;
    p.lds = lds;
    p.D = D;
    p.eps = eps;
    p.w_add = (flags & SV_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    p.row_scale = group == 0;
    return norm_call<true>(p, T, reinterpret_cast<cudaStream_t>(stream));
}

int gated_delta_step(const sv_delta_rows *rows, int T, const sv_delta_rows *prev, int prev_T,
                     const int32_t *accept_len, int B, const sv_delta_shape *shape, float *state,
                     const int32_t *state_idx, int n_slots, sv_bf16 *o, long long ldo, sv_stream stream)
{
    using namespace sv;
    int rc = check_delta_shape(shape);
    if (rc != SV_OK) return rc;
    if (shape->flags & SV_DELTA_ZERO_INIT) return SV_ERR_SHAPE;
    if (T < 0 || T > GD_MAX_ROWS || prev_T < 0 || prev_T > GD_MAX_ROWS) return SV_ERR_SHAPE;
    if (T > 0 && (rc = check_delta_rows(rows, shape, true)) != SV_OK) return rc;
    if (T > 0 && (rc = check_delta_out(shape, o, ldo)) != SV_OK) return rc;
    if (prev_T > 0 && (rc = check_delta_rows(prev, shape, false)) != SV_OK) return rc;
    if (!aligned_to(accept_len, 4)) return SV_ERR_ALIGN;
    rc = check_delta_state(shape, state, state_idx, n_slots, B);
    if (rc != SV_OK) return rc;
    if (B == 0 || T + prev_T == 0) return SV_OK;
    DeviceInfo dev;
    rc = ops_device(&dev);
    if (rc != SV_OK) return rc;
    DeltaParams p = delta_params(rows, shape, state, state_idx, n_slots, o, ldo, dev);
    p.T = T;
    p.prev_T = prev_T;
    if (prev_T > 0) p.prev = delta_rows(prev);
    p.accept_len = accept_len;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool split = delta_step_split(static_cast<long long>(B) * p.Hv * p.dv, dev);
    if (!delta_step_by_rows(T + prev_T, static_cast<long long>(B) * p.Hv * p.dv, dev))
        return shape->dk == 64 ? delta_block_dispatch<64>(p, B, split, cs) : delta_block_dispatch<128>(p, B, split, cs);
    const dim3 grid(static_cast<unsigned>(p.dv / GD_COLS), static_cast<unsigned>(p.Hv), static_cast<unsigned>(B));
    const int cap = T > prev_T ? T : prev_T;
    const size_t smem = 4 * static_cast<size_t>(gd_smem_floats(cap, shape->dk));
    return shape->dk == 64 ? launch(gated_delta_step_kernel<64>, grid, GD_THREADS, smem, cs, p)
                           : launch(gated_delta_step_kernel<128>, grid, GD_THREADS, smem, cs, p);
}

size_t gated_delta_chunk_bytes(int R, int B, const sv_delta_shape *shape)
{
    if (sv::check_delta_shape(shape) != SV_OK || R < 0 || B < 0) return 0;
    if (sv::delta_by_rows(R, B)) return 16;
    return sv::DC_FLAGS + sv::delta_block_bytes(R, B, shape->Hv) + 4 * (static_cast<size_t>(B) + 1);
}

int gated_delta_chunk(const sv_delta_rows *rows, int R, const int32_t *cu_seqlens, int B, const sv_delta_shape *shape,
                      float *state, const int32_t *state_idx, int n_slots, sv_bf16 *o, long long ldo, void *ws,
                      size_t ws_bytes, sv_stream stream)
{
    using namespace sv;
    int rc = check_delta_shape(shape);
    if (rc != SV_OK) return rc;
    if (shape->flags & SV_DELTA_COMMIT) return SV_ERR_SHAPE;
    // (a kernel counts the heads' blocks, and DS_EXTRA more a sequence, in 32 bits)
    if (R < 0 || (delta_blocks(R, B) + 1LL * DS_EXTRA * B) * shape->Hv > 0x7FFFFFFF) return SV_ERR_SHAPE;
    if (R > 0 && (rc = check_delta_rows(rows, shape, true)) != SV_OK) return rc;
    if (R > 0 && (rc = check_delta_out(shape, o, ldo)) != SV_OK) return rc;
    rc = check_delta_state(shape, state, state_idx, n_slots, B);
    if (rc != SV_OK) return rc;
    if (!cu_seqlens || !ws) return SV_ERR_NULL;
    if (!aligned_to(cu_seqlens, 4) || !aligned_to(ws, 16)) return SV_ERR_ALIGN;
    if (ws_bytes < gated_delta_chunk_bytes(R, B, shape)) return SV_ERR_SHAPE;
    if (B == 0) return SV_OK;
    DeviceInfo dev;
    rc = ops_device(&dev);
    if (rc != SV_OK) return rc;
    DeltaChunkParams p{};
    p.d = delta_params(rows, shape, state, state_idx, n_slots, o, ldo, dev);
    p.cu = cu_seqlens;
    p.R = R;
    p.B = B;
    p.flags = static_cast<unsigned *>(ws);
    p.blocks = static_cast<uint8_t *>(ws) + DC_FLAGS;
    p.cu_run = reinterpret_cast<int32_t *>(p.blocks + delta_block_bytes(R, B, shape->Hv));
    p.zero_init = (shape->flags & SV_DELTA_ZERO_INIT) != 0;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (!delta_by_rows(R, B)) return shape->dk == 64 ? delta_chunk_launch<64>(p, dev, cs) : delta_chunk_launch<128>(p, dev, cs);
    const dim3 grid(static_cast<unsigned>(p.d.dv / GD_COLS), static_cast<unsigned>(p.d.Hv), static_cast<unsigned>(B));
    const size_t smem = 4 * static_cast<size_t>(gd_smem_floats(GD_MAX_ROWS, shape->dk));
    static_assert(4 * gd_smem_floats(GD_MAX_ROWS, 128) <= 48 * 1024, "no launch needs the limit raised");
    return shape->dk == 64 ? launch(gated_delta_rows_kernel<64>, grid, GD_THREADS, smem, cs, p)
                           : launch(gated_delta_rows_kernel<128>, grid, GD_THREADS, smem, cs, p);
}

int w4a16_gate_up(const sv_bf16 *x, const uint32_t *Wq, const sv_bf16 *scales, int T, int K, int F, int act,
                  sv_bf16 *h, sv_stream stream)
{
    using namespace sv;
    if (!x || !Wq || !scales || !h) return SV_ERR_NULL;
    if (T < 1 || T > GU_MAX_TOKENS || K < 128 || K % 128 || F < 1 || F > (1 << 30)) return SV_ERR_SHAPE;
    if (act != SV_ACT_SILU && act != SV_ACT_GELU_TANH) return SV_ERR_SHAPE;
    if (!aligned_to(x, 16) || !aligned_to(Wq, 16) || !aligned_to(scales, 16) || !aligned_to(h, 16)) return SV_ERR_ALIGN;
    DeviceInfo dev;
    const int rc = ops_device(&dev);
    if (rc != SV_OK) return rc;
    GateUpParams p{};
    p.x = x;
    p.Wq = Wq;
    p.scales = scales;
    p.h = h;
    p.T = T;
    p.K = K;
    p.G = K / 128;
    p.F = F;
    p.tiles = (F + 7) / 8;
    p.act = act;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (gate_up_wide(T, p.G, gate_up_cols(F, dev.sms)))
        return T <= 16 ? gate_up_tc_launch<16>(p, dev, cs) : gate_up_tc_launch<32>(p, dev, cs);
    const int per = (p.tiles + dev.sms - 1) / dev.sms;      // tiles of a block
    while (p.ks_log < 4 && (per << (p.ks_log + 1)) <= GU_WARPS) ++p.ks_log;
    if (T <= 8) return gate_up_launch<1>(p, dev, cs);
    if (T <= 16) return gate_up_launch<2>(p, dev, cs);
    return gate_up_launch<4>(p, dev, cs);
}

}  // extern "C"
