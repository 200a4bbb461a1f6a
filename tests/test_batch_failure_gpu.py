"""The batched kernels' way out of a pipeline that broke, without a GPU fault:
waits that give up within a limit, and the calls after them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_the_lanes_of_a_warp_leave_a_broken_wait_together(cuda_lib):
    """Whether a wait's barrier or the block's abort came first is one answer for the warp, however its lanes poll."""
    assert cuda_lib.attn_get_status() == 0
    lanes = torch.full((8,), 7, dtype=torch.int32, device="cuda")
    for us in (50, 200, 1000, 3000) * 10:
        lanes.fill_(7)
        cuda_lib.attn_selftest_warp_wait(lanes, us)
        assert cuda_lib.attn_get_status() == cuda_lib.ATTN_ERR_TIMEOUT
        got = [x & 0xffffffff for x in lanes.tolist()]
        assert got[0] == 0 and all(x in (0, 0xffffffff) for x in got), got
    for bad in (0, 2000000):
        with pytest.raises(cuda_lib.AttnError):
            cuda_lib.attn_selftest_warp_wait(lanes, bad)
    assert cuda_lib.attn_get_status() == 0
