// selftest.cu -- exercises the kernels' failure path on purpose: one CTA
// waits, with the same bounded-wait routine every kernel uses, on an mbarrier
// that nothing will ever complete.  The wait gives up after the requested
// limit, the kernel records ATTN_ERR_TIMEOUT in the status word and returns;
// no fault, no hang, and the CUDA context stays usable.  A second test runs
// both forms of the warp-wide wait of the batched kernels into the same end.
#include "../../include/attn_gqa.h"
#include "batch.h"
#include "batch_wait.cuh"
#include "common.cuh"
#include "internal.h"

namespace attn {
namespace {

__global__ void wait_never_kernel(unsigned* status, unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);  // one arrival expected; none will come
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  mbar_wait_bounded(&bar, 0, status, &abort_flag, limit_ns);
}

// Warp 0's wait gives up, which sets the abort flag, and then the barrier that
// the other warps wait for completes: their lanes, which began to wait one
// after the other, see either first.  lanes[w] = the lanes of warp w whose wait
// succeeded.
constexpr int kWaitWarps = 8;
template <bool SHORT>
__global__ void warp_wait_kernel(unsigned* status, unsigned* lanes, unsigned long long limit_ns) {
  __shared__ uint64_t never, late;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&never, 1);
    mbar_init(&late, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  bool ok;
  if (warp == 0) {
    ok = warp_wait<false, SHORT>(&never, 0, status, &abort_flag, limit_ns);
    if (lane == 0) mbar_arrive(&late);
  } else {
    __nanosleep(lane * 100);
    ok = warp_wait<false, SHORT>(&late, 0, status, &abort_flag);
  }
  const unsigned mask = __ballot_sync(0xffffffffu, ok);
  if (lane == 0) lanes[warp] = mask;
}

}  // namespace
}  // namespace attn

extern "C" int attn_selftest_wait_timeout(uint32_t timeout_us, attn_stream_t stream) {
  if (timeout_us == 0 || timeout_us > 1000000u) return ATTN_ERR_INVALID_ARG;
  unsigned* st = attn::device_status_word();
  if (st == nullptr) return ATTN_ERR_CUDA;
  attn::wait_never_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      st, (unsigned long long)timeout_us * 1000ull);
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_selftest_batch_wait(uint32_t limit_ns) {
  if (limit_ns > attn::kWaitLimitNs) return ATTN_ERR_INVALID_ARG;
  attn::set_batch_wait_ns(limit_ns);
  return ATTN_OK;
}

template <bool SHORT>
static int selftest_warp_wait(uint32_t timeout_us, uint32_t* lanes, attn_stream_t stream) {
  if (timeout_us == 0 || timeout_us > 1000000u || lanes == nullptr) return ATTN_ERR_INVALID_ARG;
  unsigned* st = attn::device_status_word();
  if (st == nullptr) return ATTN_ERR_CUDA;
  attn::warp_wait_kernel<SHORT><<<1, 32 * attn::kWaitWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      st, lanes, (unsigned long long)timeout_us * 1000ull);
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int attn_selftest_warp_wait(uint32_t timeout_us, uint32_t* lanes, attn_stream_t stream) {
  return selftest_warp_wait<false>(timeout_us, lanes, stream);
}

extern "C" int attn_selftest_short_wait(uint32_t timeout_us, uint32_t* lanes, attn_stream_t stream) {
  return selftest_warp_wait<true>(timeout_us, lanes, stream);
}
