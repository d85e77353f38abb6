// op_launch.h -- what the calls without a context need to know of the device
// and of a kernel before a launch, kept for the life of the process: such a
// call is issued for every decoded token, and each question to the runtime
// costs it a fraction of a microsecond.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace cam {

constexpr int kMaxSharedBytes = 227 * 1024;  // dynamic shared memory a block may have
constexpr int kMaxDevices = 64;

// The current device and its SM count.
inline cudaError_t current_device(int* dev, int* sms) {
    static std::atomic<int> known[kMaxDevices];
    cudaError_t ce = cudaGetDevice(dev);
    if (ce != cudaSuccess) return ce;
    const bool keep = *dev < kMaxDevices;
    *sms = keep ? known[*dev].load(std::memory_order_relaxed) : 0;
    if (*sms > 0) return cudaSuccess;
    ce = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (ce == cudaSuccess && keep) known[*dev].store(*sms, std::memory_order_relaxed);
    return ce;
}

// Lets a kernel have up to kMaxSharedBytes on device `dev`; `done` is the
// kernel's own record of the devices where it may.
inline cudaError_t allow_shared(const void* kernel, int dev, std::atomic<uint64_t>& done) {
    const uint64_t bit = dev < kMaxDevices ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t ce =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSharedBytes);
    if (ce == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return ce;
}

}  // namespace cam
