// resident.cuh -- how many CTAs of a kernel the current device holds at once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

constexpr int kResidentDevices = 64;

// Queried once per kernel (the template's instance) and device; a race writes the same value twice.
template <typename... KArgs>
inline cudaError_t resident_ctas_at(int64_t (&cached)[kResidentDevices], void (*kernel)(KArgs...), int threads,
                                    size_t smem, int64_t &out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < kResidentDevices;
    if (keep && cached[dev] > 0) {
        out = cached[dev];
        return cudaSuccess;
    }
    int per_sm = 0, sms = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (per_sm < 1 || sms < 1) return cudaErrorInvalidConfiguration;
    out = (int64_t)per_sm * sms;
    if (keep) cached[dev] = out;
    return cudaSuccess;
}

}  // namespace ssd
