// launch.h -- kernel launches with programmatic dependent launch enabled: the grid may
// be scheduled while the previous work on the stream is still running, and its
// kernel calls pdl_wait() (ptx.cuh) before reading anything that work produced.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace mha {

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// launch_pdl with clusters of `size` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, int size, size_t smem, cudaStream_t s,
                               Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(size), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// SMs of the current device.
inline cudaError_t sm_count(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Clusters of a kernel, allowed `smem` bytes by the caller, that the current device runs at once; asked once a device and
// size, for it is a property of the device.
struct ClusterRoom {
    static constexpr int kDevices = 64;
    std::atomic<int> known[kDevices][5] = {};      // by log2(size); 0: not asked, else 1 + the answer
    template <typename Kernel>
    int at_once(Kernel kernel, int threads, size_t smem, int size) {
        const int lg = size == 16 ? 4 : size == 8 ? 3 : size == 4 ? 2 : 1;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
        if (const int k = known[dev][lg].load(std::memory_order_relaxed)) return k - 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {static_cast<unsigned>(size), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
        known[dev][lg].store(n + 1, std::memory_order_relaxed);
        return n;
    }
};

}  // namespace mha
