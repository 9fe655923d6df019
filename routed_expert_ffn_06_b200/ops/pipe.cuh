// pipe.cuh -- waits of the operators' pipelines (shared-memory rings, TMEM
// accumulators).
#pragma once
#include "common.cuh"

namespace moe {

// A wait of a running pipeline.  The lanes of a warp do not vote on the outcome (a
// vote costs about 60 cycles, as much as the wait itself) and may leave it apart:
// instructions of the whole warp come after a __syncwarp(), which costs nothing
// measurable (8192 x 4096 x 2048 73.2 us with and without).
//
// A wait that runs out (moe.h's limit; the timer is only read after kPolls polls)
// records the error and raises the block's `gave_up` flag, and from then on every
// wait of the block that is not over soon returns false.  The lane that issues
// copies or MMAs stops for good at its first false wait; the warps walk their loops
// to the end on whatever the memory holds, so the outputs are undefined.  At most
// one ring of copies is in flight then, each on the newest phase of its stage's
// barrier, and pipe_drain waits for those.
constexpr int kPolls = 4096;
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity, Control* ctl,
                                          uint32_t where, uint32_t* gave_up) {
  if (mbar_try_wait(bar, parity)) return true;
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*reinterpret_cast<volatile uint32_t*>(gave_up)) return false;
      if (i >= kPolls) {
        const bool ok = mbar_wait(bar, parity, ctl, where);
        if (!ok) *reinterpret_cast<volatile uint32_t*>(gave_up) = 1u;
        return ok;
      }
    }
  }
}

// The lane that issued n fills of a ring of `stages` barriers waits for the newest
// of each stage: nobody may have consumed them, and no copy may outlive the block.
// They complete on their bytes alone, so these waits do not mind gave_up.
__device__ __forceinline__ void pipe_drain(uint64_t* full, int stages, long long n, Control* ctl,
                                           uint32_t where) {
  for (long long j = n > stages ? n - stages : 0; j < n; ++j)
    mbar_wait(&full[j % stages], (uint32_t)(j / stages) & 1u, ctl, where);
}

}  // namespace moe
