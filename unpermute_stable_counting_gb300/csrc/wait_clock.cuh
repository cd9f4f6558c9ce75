// How long a wait has been going on, for kernels that give a wait up after a
// while: the time between readings that follow one another closely. A context that
// is not running (suspended by a debugger, or in favour of another process) reads
// no clock; what passes meanwhile is no sign of a copy that does not come, and
// counts as kGap at most. Plain C++, so that it is tested without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MR_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MR_HOST_DEVICE inline
#endif

namespace mr {

struct WaitClock {
    static constexpr uint32_t kGap = 100000000u / 1024u;  // 0.1 s in units of 1024 ns: far above what 64 polls take
    static constexpr uint32_t kLimit = 20u * kGap;

    uint32_t last = 0u, waited = 0u;
    bool started = false;

    // A reading of the clock, in ns: whether the wait has reached its limit. The
    // first one starts the wait, and at least 20 more come up to the limit.
    MR_HOST_DEVICE bool out(uint64_t ns) {
        const uint32_t now = (uint32_t)(ns >> 10), gap = started ? now - last : 0u;
        started = true;
        last = now;
        waited += gap < kGap ? gap : kGap;
        return waited >= kLimit;
    }
};

}  // namespace mr
