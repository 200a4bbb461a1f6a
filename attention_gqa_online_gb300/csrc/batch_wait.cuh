// batch_wait.cuh -- the bounded barrier waits of the batched attention kernels.
#pragma once

#include "common.cuh"

namespace attn {

// Waits for phase `parity` of `bar`, within limit_ns (as mbar_wait_bounded).
// The thread suspends in try_wait itself: the form with a time hint becomes a
// polling loop with sleeps, whose wake-ups come late (SYNCS and NANOSLEEP were
// a tenth of all instructions); polling with test_wait takes 8% longer.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag,
                                           unsigned long long limit_ns = kWaitLimitNs) {
  unsigned long long t0 = 0;
  for (unsigned n = 0;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if (n % 16 == 15) {
      if (*abort_flag != 0) return false;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        record_status(status, ATTN_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// The same for a warp, all of whose lanes call it together.  The lanes see a
// phase complete, or the block's abort flag set, at different times, so they
// meet again here, with one answer for all, before any of them arrives
// somewhere for the warp, takes part in a warp-wide instruction or leaves.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag,
                                          unsigned long long limit_ns = kWaitLimitNs) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, status, abort_flag, limit_ns));
}
// Is the block's pipeline whole?  One answer for the warp, too.
__device__ __forceinline__ bool warp_whole(volatile int* abort_flag) {
  return __all_sync(0xffffffffu, *abort_flag == 0);
}

}  // namespace attn
