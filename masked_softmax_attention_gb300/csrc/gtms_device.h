// gtms_device.h -- what launches need to know of the current device.
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace gtms {

// What a launch needs to know once per device and process, and never changes:
// the number of multiprocessors, and that the kernel may use `smem` bytes of
// dynamic shared memory and, where it wants them, run in clusters of more than
// eight CTAs. Devices from 64 on ask every time.
inline int device_sms()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    if (dev < 64 && known[dev].load(std::memory_order_relaxed) > 0)
        return known[dev].load(std::memory_order_relaxed);
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    if (dev < 64)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <auto Kernel, bool LargeClusters = false>
inline cudaError_t allow_smem(int smem)
{
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed)))
        return e;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && LargeClusters)
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64)
        done[dev].store(true, std::memory_order_relaxed);
    return e;
}

}  // namespace gtms
