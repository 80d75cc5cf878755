// Host-side helpers shared by the C-ABI sources: the calling thread's error
// message, NVTX ranges, sizes, and the per-device shared-memory limit.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stddef.h>
#include <stdint.h>

#include "vscan.h"
#include "vscan_route.cuh"

struct vscan_route {
    vscan::RouteGeom g;
};

namespace vscan_host {

// A named NVTX range for the duration of a public call, so a profiler's
// timeline groups each call's copies and kernels (a no-op unless a tool is
// attached; NVTX v3 is header-only).
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// Record the calling thread's message for vscan_last_error() and return s.
vscan_status fail(vscan_status s, const char* fmt, ...);
vscan_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

inline size_t elem_bytes(int32_t dtype) { return dtype == VSCAN_BF16 ? 2 : 4; }

// Raise a kernel's dynamic shared-memory limit once per device (the attribute
// stays set for the process), not on every launch: one flag per instantiation
// of the calling template and device ordinal.
template <typename Kernel>
cudaError_t set_smem_once(Kernel* fn, int bytes, int* done_by_device, int max_devices)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < max_devices && __atomic_load_n(&done_by_device[dev], __ATOMIC_ACQUIRE) >= bytes)
        return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < max_devices)
        __atomic_store_n(&done_by_device[dev], bytes, __ATOMIC_RELEASE);
    return e;
}

// Launch a kernel; with `after`, one that follows another of the same call on the stream: its blocks
// may come before that one has ended (programmatic dependent launch) and have to wait for its end
// themselves. Saves the launch latency between the kernels of small calls.
template <typename... P>
cudaError_t launch_after(bool after, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, P... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&config, kernel, args...);
}

}  // namespace vscan_host
