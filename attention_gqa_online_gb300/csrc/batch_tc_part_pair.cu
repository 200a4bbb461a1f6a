// batch_tc_part_pair.cu -- the tensor-core batched attention for head dimensions
// between 64 and 128 on pairs of multiprocessors.
#include "batch_tc.cuh"

namespace attn {

int launch_batch_tc_part_pair(const BatchArgs& a, int dtype, int blocks, int box_rows, cudaStream_t s) {
  return dtype == ATTN_DT_BF16 ? launch_tc_t<__nv_bfloat16, 128, true, false, false>(a, blocks, box_rows, s)
                               : launch_tc_t<__half, 128, true, false, false>(a, blocks, box_rows, s);
}

}  // namespace attn
