// batch_tc_sinks64.cu -- the tensor-core batched attention with first positions
// behind a window, for head dimensions up to 64.
#include "batch_tc.cuh"

namespace attn {

int launch_batch_tc_sinks64(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s) {
  return dtype == ATTN_DT_BF16 ? launch_tc_t<__nv_bfloat16, 64, false, false, true>(a, blocks, box_rows, s)
                               : launch_tc_t<__half, 64, false, false, true>(a, blocks, box_rows, s);
}

}  // namespace attn
