// Bulk copies of rows into shared memory, and the bounded wait for them.
#pragma once
#include "sc_tma.cuh"

namespace scg {

// Shared memory that a launch may ask for without a limit set for its kernel (with room
// for what the kernels have by themselves).
constexpr int kDefaultShared = 40 * 1024;

// `bytes` (a multiple of 16, both addresses aligned so) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(to), "l"(from), "r"(bytes), "r"(bar) : "memory");
}

// Copies end by themselves; a wait that should run out all the same (a second or so) gives
// up, and the caller makes NaN of what was to come of them.
__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < (1 << 20); ++i)
        if (mbar_try_wait_sleep(bar, parity, 1000)) return true;
    return false;
}

__device__ __forceinline__ float not_a_number() { return __int_as_float(0x7fffffff); }

}  // namespace scg
