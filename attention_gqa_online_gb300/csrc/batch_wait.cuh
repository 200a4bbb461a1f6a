// batch_wait.cuh -- the bounded barrier wait of the batched attention kernels.
#pragma once

#include "common.cuh"

namespace attn {

// Waits for phase `parity` of `bar`, within kWaitLimitNs (as mbar_wait_bounded).
// The thread suspends in try_wait itself: the form with a time hint becomes a
// polling loop with sleeps, whose wake-ups come late (SYNCS and NANOSLEEP were
// a tenth of all instructions).  REMOTE: the other block's threads arrive.
template <bool REMOTE>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag) {
  unsigned long long t0 = 0;
  for (unsigned n = 0;; ++n) {
    unsigned ok;
    if (REMOTE)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
    else
      ok = mbar_try_wait(bar, parity);
    if (ok) return true;
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
