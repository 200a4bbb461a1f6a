// find_seq.cuh -- the sequence of a token row.
#pragma once

#include <cstdint>

namespace attn {
namespace {

// Last s in [0, n) with starts[s] <= row, or -1; every lane gets the result.
__device__ __forceinline__ int find_seq(const uint32_t* starts, int n, uint32_t row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the answer, if any, is in [lo, hi)
  while (true) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && starts[at] <= row;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    if (step == 1) return lo;
    hi = min(hi, lo + step);
  }
}

}  // namespace
}  // namespace attn
