// waiter.cuh -- the bounded mbarrier wait every role of the pipelined kernels
// uses: a time limit, the CTA's abort flag, and the status word a wait that
// gives up is recorded in.
#pragma once

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace pws {

// Bounded mbarrier wait.  Returns false if the wait gave up (time limit or
// another role's abort); the first role to give up records the timeout.
struct Waiter {
    unsigned long long timeout_ns;
    volatile uint32_t* abort;
    unsigned* status;
    unsigned role;

    template <bool CLUSTER_SCOPE = false>
    __device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity) const {
        return CLUSTER_SCOPE ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
    }

    __device__ __forceinline__ bool give_up() const {
        *abort = 1u;
        atomicOr(status, kStatusTimeout | role);
        return false;
    }

    // A wait that lasts about one K block (the ring's, the accumulator
    // hand-over's): the limit counts from the start of the wait.
    template <bool CLUSTER_SCOPE = false>
    __device__ bool wait(uint32_t bar, uint32_t parity) const {
        return wait_inline<CLUSTER_SCOPE>(bar, parity);
    }

    // The same, inlined into the caller: for a caller holding many registers
    // across the wait (the realigning producer's loads in flight).
    template <bool CLUSTER_SCOPE = false>
    __device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity) const {
        if (probe<CLUSTER_SCOPE>(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (probe<CLUSTER_SCOPE>(bar, parity)) return true;
            if (*abort) return false;
            if (globaltimer_ns() - t0 > timeout_ns) return give_up();
        }
    }

    // A wait that legitimately lasts a whole K loop: the epilogue's wait for
    // a finished accumulator, and the K split's wait for the peer's partial
    // sums.  The limit counts from the last change of the progress counter
    // that the producer of the CTA being waited for bumps once per K block
    // (`remote`: the counter lives in the other CTA of the cluster), so such
    // a wait gives up on a stall -- no K block issued for the whole limit --
    // and never on a long but live loop.  After the producer's last block the
    // wait still has to cover at most S blocks of multiplies and a drain.
    template <bool CLUSTER_SCOPE = false>
    __device__ bool wait_progress(uint32_t bar, uint32_t parity, uint32_t progress, bool remote) const {
        if (probe<CLUSTER_SCOPE>(bar, parity)) return true;
        uint64_t t0 = globaltimer_ns();
        uint32_t seen = remote ? ld_relaxed_cluster_u32(progress) : ld_volatile_shared_u32(progress);
        for (;;) {
            if (probe<CLUSTER_SCOPE>(bar, parity)) return true;
            if (*abort) return false;
            const uint32_t now_seen = remote ? ld_relaxed_cluster_u32(progress) : ld_volatile_shared_u32(progress);
            const uint64_t now = globaltimer_ns();
            if (now_seen != seen) {
                seen = now_seen;
                t0 = now;
            } else if (now - t0 > timeout_ns) {
                return give_up();
            }
        }
    }
};

}  // namespace pws
