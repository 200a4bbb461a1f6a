// batch_wait.cuh -- the bounded barrier wait of the batched attention kernels.
#pragma once

#include "common.cuh"

namespace attn {

// Waits for phase `parity` of `bar`, within kWaitLimitNs (as mbar_wait_bounded).
// The thread suspends in try_wait itself: the form with a time hint becomes a
// polling loop with sleeps, whose wake-ups come late (SYNCS and NANOSLEEP were
// a tenth of all instructions); polling with test_wait takes 8% longer.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag) {
  unsigned long long t0 = 0;
  for (unsigned n = 0;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if (n % 16 == 15) {
      if (*abort_flag != 0) return false;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        record_status(status, ATTN_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

}  // namespace attn
