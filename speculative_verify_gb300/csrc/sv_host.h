// sv_host.h -- what the library's translation units share on the host: the
// per-device facts and the sticky error word kept by specverify.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sv {

struct DeviceInfo {
    int dev;            // the current device's ordinal
    int sms;            // multiprocessors
    int smem_optin;     // largest dynamic shared memory of a block, bytes
    int *err;           // sticky device error word
};

// The current device's facts; creates the device's scratch area on first
// use, as every entry point does.  SV_OK or a negative status.
int device_info(DeviceInfo *out);

inline bool aligned_to(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A launch configuration with programmatic dependent launch, as every kernel
// of a verify cycle is launched; `attr` lives as long as the configuration.
inline void launch_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, dim3 grid, int threads, size_t smem,
                          cudaStream_t stream)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = grid;
    cfg->blockDim = dim3(static_cast<unsigned>(threads));
    cfg->dynamicSmemBytes = smem;
    cfg->stream = stream;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
}

}  // namespace sv
