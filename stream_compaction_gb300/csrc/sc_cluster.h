// Whether the device holds clusters of more than 8 CTAs, the size that every device has.
#pragma once
#include <atomic>
#include <cuda_runtime.h>

namespace scg {

// Asked once for each device (64 of them) with one launch configuration, the largest that a
// kernel has: some parts of a chip, or a part of it that a process is given, may have too
// few multiprocessors for a cluster, which would make its launch fail.
struct LargeClusters {
    std::atomic<unsigned long long> known{0}, held{0};
    bool fit(const void* kernel, const cudaLaunchConfig_t& cfg) {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        const unsigned long long bit = 1ull << (dev & 63);
        if (!(known.load() & bit)) {
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) cudaGetLastError();
            else if (n > 0) held.fetch_or(bit);
            known.fetch_or(bit);
        }
        return (held.load() & bit) != 0;
    }
};

}  // namespace scg
