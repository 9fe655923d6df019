// pipe.cuh -- waits of the operators' pipelines (shared-memory rings, TMEM
// accumulators) that do not leave a warp divided.
#pragma once
#include "common.cuh"

namespace moe {

// A wait of a running pipeline.  The warps that wait stay whole without voting
// on the outcome (a vote costs about 60 cycles, as much as the wait itself): a
// wait that runs out (moe.h's limit; the timer is only read after kPolls polls)
// records the error and raises the block's `gave_up` flag, and from then on
// every wait of the block returns at once.  The roles then run to their ends on
// whatever the memory holds; the outputs are undefined, but no copy outlives
// the block (pipe_drain).
constexpr int kPolls = 4096;
__device__ __forceinline__ void pipe_wait(uint64_t* bar, uint32_t parity, Control* ctl,
                                          uint32_t where, uint32_t* gave_up) {
  if (mbar_try_wait(bar, parity)) return;
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 63) == 0) {
      if (*reinterpret_cast<volatile uint32_t*>(gave_up)) return;
      if (i >= kPolls) {
        if (!mbar_wait(bar, parity, ctl, where)) *reinterpret_cast<volatile uint32_t*>(gave_up) = 1u;
        return;
      }
    }
  }
}

// Copies in flight when a block gave up may count on barriers that it can no
// longer follow: it outlives them by time.
__device__ __forceinline__ void pipe_drain(const uint32_t* gave_up) {
  if (*reinterpret_cast<const volatile uint32_t*>(gave_up)) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kWaitFloorNs) __nanosleep(1000);
  }
}

}  // namespace moe
