// batch_tc_d128.cu -- the tensor-core batched attention for head dimension 128.
#include "batch_tc.cuh"

namespace attn {

int launch_batch_tc_d128(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s) {
  return dtype == ATTN_DT_BF16 ? launch_tc_t<__nv_bfloat16, 128, false, true, false>(a, blocks, box_rows, s)
                               : launch_tc_t<__half, 128, false, true, false>(a, blocks, box_rows, s);
}

}  // namespace attn
