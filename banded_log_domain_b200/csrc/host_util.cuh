// Host-side helpers shared by the library's translation units: pointer checks,
// workspace rounding, the driver entry point for tensor maps, the SM count and
// the launch with programmatic stream serialisation.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <utility>

#include "../../include/sinkhorn_attn.h"

namespace sa {

constexpr size_t kHeader = 256;   // status word + padding at the start of every workspace

inline size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned16(const void* x) { return ((uintptr_t)x & 15u) == 0; }

// Memory the current device's kernels may read and write at full speed: device
// memory of the current device, or managed memory.  Pinned host memory (read
// over PCIe), pageable host memory, and another device's memory (a tensor on
// another GPU, or the wrong device current) are rejected before any launch.
inline bool on_current_device(const void* x) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, x) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (at.type == cudaMemoryTypeManaged) return true;
    if (at.type != cudaMemoryTypeDevice) return false;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return at.device == dev;
}
inline bool device_ok(const void* x) { return x && aligned16(x) && on_current_device(x); }
// A device float that may sit anywhere a float may (4-byte alignment).
inline bool device_f32_ok(const void* x) { return x && ((uintptr_t)x & 3u) == 0 && on_current_device(x); }
// The byte mask (any alignment; NULL means every token is valid).
inline bool mask_ok(const void* x) { return !x || on_current_device(x); }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
inline PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// SMs of the device (persistent grids take one or two CTAs per SM); read once
// from the first device asked, since the library targets a single GPU model
// (sm_100a)
inline int sm_count() {
    static int nsm = 0;
    if (nsm == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || nsm <= 0)
            nsm = 148;
    }
    return nsm;
}

// Launches a persistent sweep with programmatic stream serialisation: its
// CTAs may be placed while the previous kernel of the stream finishes, so their
// set-up (barrier init, TMEM allocation) overlaps its tail; the sweeps wait for
// that kernel (griddepcontrol.wait) before any global access, so the ordering
// of their reads and writes is that of a plain launch.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace sa
