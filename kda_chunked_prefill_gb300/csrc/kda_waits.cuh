// Bounded waits of a kernel's roles on barriers in shared memory. M: the kernel's bookkeeping in shared memory, whose `abort` says that some role has
// given up.
#pragma once
#include "kda_linear.cuh"

namespace kda {

// waits of up to 0.1 ms each before a role gives up; and before one that has given up takes its own copies for complete
constexpr int WAITS = 20000, WAITS_DRAIN = 100;

template <typename M>
__device__ __forceinline__ bool wait(M *m, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    int i = 0;
#pragma unroll 1
    while (!lin::mbar_wait_some(bar, parity)) {
        if (++i == WAITS) *reinterpret_cast<volatile int32_t *>(&m->abort) = 1;
        if (*reinterpret_cast<volatile int32_t *>(&m->abort)) return false;
    }
    return true;
}
__device__ __forceinline__ void wait_drain(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < WAITS_DRAIN && !lin::mbar_wait_some(bar, parity); ++i) {
    }
}
template <typename M>
__device__ __forceinline__ bool wait_warp(M *m, uint64_t *bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;  // (the warp stays together)
    return __all_sync(0xffffffffu, wait(m, bar, parity));
}

}  // namespace kda
