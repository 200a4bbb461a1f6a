// batch_wait.cuh -- the bounded barrier waits of the batched attention kernels.
#pragma once

#include "common.cuh"

namespace attn {

// Waits for phase `parity` of `bar`, within limit_ns (as mbar_wait_bounded).
// The thread suspends in try_wait for as long as that takes by itself: a prompt
// of 8192, 32 heads over 8 of 128, takes 399 us so, 405 with a hint of 2 us, 427
// polling with test_wait.
// BRIEF, for the failure-path test's kernels, polls and looks at the limit each
// time (chosen at run time it took 15% of a prompt's time).
template <bool BRIEF = false>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag,
                                           unsigned long long limit_ns = kWaitLimitNs) {
  unsigned long long t0 = 0;
  for (unsigned n = 0;; ++n) {
    if (BRIEF ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (BRIEF || n % 16 == 15) {
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
template <bool BRIEF = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag,
                                          unsigned long long limit_ns = kWaitLimitNs) {
  return __all_sync(0xffffffffu, wait_phase<BRIEF>(bar, parity, status, abort_flag, limit_ns));
}
// Is the block's pipeline whole?  One answer for the warp, too.
__device__ __forceinline__ bool warp_whole(volatile int* abort_flag) {
  return __all_sync(0xffffffffu, *abort_flag == 0);
}

// A tile's copies come from several issuers and complete on one barrier, armed
// by one of them for all of its bytes.  Where the pipeline broke, some may have
// issued a tile that others have not.  This lets the barrier's phase complete
// with the copies that were issued: `missing` bytes never come.
__device__ __forceinline__ void settle_tile(uint64_t* full, bool armed, unsigned bytes, unsigned missing) {
  if (armed)
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(full)), "r"(missing)
                 : "memory");
  else
    mbar_arrive_expect_tx(full, bytes - missing);
}
// Waits for the last tile of every slot of a ring into which `issued` tiles were copied.
__device__ __forceinline__ void drain_ring(uint64_t* full, int slots, int issued, unsigned* status) {
  for (int s = 0; s < slots && s < issued; ++s) {
    const int last = s + ((issued - 1 - s) / slots) * slots;
    mbar_wait_bounded(&full[s], (unsigned)((last / slots) & 1), status);
  }
}

}  // namespace attn
