// gated_delta_chunk.cuh -- the gated delta rule over whole prompts.
#pragma once

#include "gated_delta.cuh"

namespace sv {

struct DeltaChunkParams {
    DeltaParams d;                              // rows, shape, state; T and prev unused
    const int32_t *cu;                          // [B + 1] first rows
    int R;                                      // rows in all
    int zero_init;
};

// The rows of sequence b: cu[b] .. cu[b + 1], kept within [0, R].
__device__ __forceinline__ void gd_range(const int32_t *cu, int R, int b, int &begin, int &end)
{
    begin = min(max(cu[b], 0), R);
    end = min(max(cu[b + 1], begin), R);
}

// Row by row.  Grid: x = dv / cols, y = Hv, z = B.
template <int DK>
__global__ void __launch_bounds__(512) gated_delta_rows_kernel(const DeltaChunkParams cp)
{
    extern __shared__ __align__(16) float gd_smem[];
    const DeltaParams &p = cp.d;
    const int cols = p.cols, col0 = blockIdx.x * cols, hv = blockIdx.y, b = blockIdx.z;
    const int i = threadIdx.x & 3, col = threadIdx.x >> 2;
    const GdSmem<DK> sm(gd_smem, GD_MAX_ROWS, cols);
    pdl_launch_dependents();
    pdl_wait_prior();
    int begin, end;
    gd_range(cp.cu, cp.R, b, begin, end);
    const int slot = gd_slot(p.state_idx, p.n_slots, b, p.err);
    uint16_t *o = p.o + begin * p.ldo + static_cast<long long>(hv) * p.dv + col0;
    if (slot < 0) {
        for (int t = begin; t < end; ++t, o += p.ldo)
            if (i == 0) o[col] = 0;
        return;
    }
    float *s = p.state + ((static_cast<long long>(slot) * p.Hv + hv) * p.dv + col0 + col) * DK;
    GdState<DK> st;
    if (cp.zero_init)
        st.zero();
    else
        st.load(s, i);
    for (int r0 = begin; r0 < end; r0 += GD_MAX_ROWS) {
        const int n = min(GD_MAX_ROWS, end - r0);
        const bool running = gd_stage<DK>(p, p.rows, r0, n, hv, col0, cols, sm, true);
        gd_rows<DK, true>(st, sm, n, cols, running, o, p.ldo);
        o += n * p.ldo;
        __syncthreads();
    }
    st.store(s, i);
}

}  // namespace sv
