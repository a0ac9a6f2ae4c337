// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace mla {

// SMs of the current device.
inline bool sm_count(int* sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && *sms >= 2)
        return true;
    cudaGetLastError();
    return false;
}

// Runs a per-device set-up step (a kernel attribute) once for each device it is used on,
// from any number of host threads.
struct PerDeviceOnce {
    static constexpr int kMaxDevices = 64;
    std::mutex m;
    std::atomic<bool> done[kMaxDevices] = {};

    template <typename F>
    cudaError_t run(F&& setup)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return setup();  // outside the table: every call
        if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
        std::lock_guard<std::mutex> lock(m);
        if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
        e = setup();
        if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
        return e;
    }
};

// Launch configuration with programmatic stream serialization: the grid may start
// while the previous one in the stream finishes; each kernel calls
// grid_dependency_wait() before it reads global memory that grid could have written.
inline void programmatic_launch(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, dim3 grid, dim3 block,
                                size_t smem, cudaStream_t stream)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
}

}  // namespace mla
