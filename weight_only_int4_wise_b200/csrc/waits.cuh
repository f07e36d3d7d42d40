// Bounded waits on mbarrier phases, shared by the tensor-core kernels. A wait
// that runs out latches W4A16_ERR_TIMEOUT in the kernel's status word.
#pragma once

#include <cstdint>

#include "../../include/w4a16.h"
#include "ptx.cuh"

namespace w4a16 {

constexpr long long kTimeoutCycles = 4000000000ll;  // about 2 s per wait at the boost clock

// Bounded wait on an mbarrier phase. Returns false if the CTA is aborting or
// the wait ran out (which starts the abort). The bound is counted in SM clock
// cycles (clock64 is a cheap, SM-local register; the global timer is far slower
// to read and would add its latency to every pipeline hand-off).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit,
                                           int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    long long start = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 0) {
            if (*abort_flag) return false;
            const long long now = clock64();
            if (start == 0) {
                start = now;
            } else if (now - start > limit) {
                *abort_flag = 1;
                atomicCAS(status, 0, W4A16_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

// Bounded wait that ignores the abort flag: used where in-flight asynchronous
// work must finish before its resources are released.
__device__ __forceinline__ bool drain_phase(uint64_t* bar, uint32_t parity, int* status) {
    const long long limit = kTimeoutCycles;  // drains keep the long bound whatever the wait bound is
    long long start = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 15u) {
            const long long now = clock64();
            if (start == 0) {
                start = now;
            } else if (now - start > limit) {
                atomicCAS(status, 0, W4A16_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

// Warp-collective forms: lane 0 polls (so the timeout decision is the same for
// the whole warp), then every lane observes the completed phase itself, which
// gives each lane acquire ordering on the data the phase guards. The phase
// cannot move on before this warp arrives elsewhere, so that check is immediate.
__device__ __forceinline__ bool warp_wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                long long limit, int* status) {
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = wait_phase(bar, parity, abort_flag, limit, status) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) mbar_try_wait(bar, parity);
    return ok != 0;
}

__device__ __forceinline__ bool warp_drain_phase(uint64_t* bar, uint32_t parity, int* status) {
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = drain_phase(bar, parity, status) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) mbar_try_wait(bar, parity);
    return ok != 0;
}

}  // namespace w4a16
