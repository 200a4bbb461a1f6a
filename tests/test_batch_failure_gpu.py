"""The batched kernels' way out of a pipeline that broke, without a GPU fault:
waits that give up within a limit, and the calls after them."""
import pytest
import torch

from batch_ref import Batch

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


@pytest.fixture
def brief_waits(cuda_lib):
    """Sets the limit of the waits inside the batched kernels; the usual one is back at the end."""
    yield cuda_lib.attn_selftest_batch_wait
    cuda_lib.attn_selftest_batch_wait(0)


# One batch per kernel and form: single tokens (whole and part heads, split and whole items), tcgen05 on single
# multiprocessors and on pairs (Q as boxes and by a warp).
BROKEN = [
    dict(H=32, G=8, D=128, new=[1] * 40, kv=[3000] * 40),
    dict(H=32, G=8, D=128, new=[1], kv=[9000]),
    dict(H=14, G=2, D=64, new=[1, 1, 1], kv=[5000, 30, 800], softcap=30.0),
    dict(H=8, G=8, D=96, new=[1] * 9, kv=[700] * 9),
    dict(H=8, G=2, D=64, new=[300, 2], kv=[4000, 900]),
    dict(H=10, G=2, D=64, new=[300, 2], kv=[4000, 900]),
    dict(H=8, G=2, D=40, new=[300, 2], kv=[4000, 900]),
    dict(H=32, G=8, D=128, new=[8, 1, 4], kv=[9000, 70, 300]),
    dict(H=32, G=8, D=96, new=[8, 1, 4], kv=[9000, 70, 300]),
    dict(H=32, G=8, D=128, new=[700, 256], kv=[4000, 256]),
    dict(H=16, G=16, D=128, new=[700, 600], kv=[2000, 600]),
    dict(H=32, G=8, D=96, new=[700, 256], kv=[4000, 256]),
]


@pytest.mark.parametrize("case", BROKEN, ids=lambda c: "H%d-G%d-D%d-%d" % (c["H"], c["G"], c["D"], sum(c["new"])))
def test_calls_whose_waits_run_out_end_and_leave_later_calls_right(cuda_lib, brief_waits, case):
    """Waits of ordinary calls run out within nanoseconds to tens of microseconds, wherever the pipeline is then: each
    call ends, with ATTN_ERR_TIMEOUT or a result, and the next call on a fresh workspace has its usual bits."""
    A, kw = cuda_lib, dict(case)
    b = Batch(kw.pop("new"), kw.pop("kv"), kw.pop("H"), kw.pop("G"), kw.pop("D"), 32, torch.bfloat16, seed=71)
    want = A.attend_paged(b.object(A), b.q, b.k, b.v, **kw)
    assert A.attn_get_status() == 0
    ran_out = 0
    for ns in (1, 100, 300, 1000, 3000, 10000, 30000) * 4:
        brief_waits(ns)
        got = A.attend_paged(b.object(A), b.q, b.k, b.v, **kw)
        status = A.attn_get_status()
        brief_waits(0)
        assert status in (0, A.ATTN_ERR_TIMEOUT)
        assert status or torch.equal(got, want)
        ran_out += status != 0
        again = A.attend_paged(b.object(A), b.q, b.k, b.v, **kw)
        assert A.attn_get_status() == 0 and torch.equal(again, want)
    assert ran_out


@pytest.mark.parametrize("case", BROKEN, ids=lambda c: "H%d-G%d-D%d-%d" % (c["H"], c["G"], c["D"], sum(c["new"])))
def test_a_workspace_serves_on_after_a_call_whose_waits_ran_out(cuda_lib, brief_waits, case):
    """A broken call leaves pieces of split items uncounted; the next calls on its workspace must not count on them."""
    A, kw = cuda_lib, dict(case)
    b = Batch(kw.pop("new"), kw.pop("kv"), kw.pop("H"), kw.pop("G"), kw.pop("D"), 32, torch.bfloat16, seed=72)
    obj = b.object(A)
    want = A.attend_paged(obj, b.q, b.k, b.v, **kw)
    for ns in (100, 1000, 2000, 4000, 8000, 16000) * 4:
        brief_waits(ns)
        A.attend_paged(obj, b.q, b.k, b.v, **kw)
        assert A.attn_get_status() in (0, A.ATTN_ERR_TIMEOUT)
        brief_waits(0)
        for _ in range(2):
            again = A.attend_paged(obj, b.q, b.k, b.v, **kw)
            assert A.attn_get_status() == 0 and torch.equal(again, want)


def test_counts_left_in_the_workspace_do_not_reach_a_later_call(cuda_lib):
    """As above, with the counts of a broken call written by hand: one piece of every item seen."""
    A = cuda_lib
    for new, kv in (([1], [9000]), ([8], [9000]), ([300], [6000])):
        b = Batch(new, kv, 32, 8, 128, 32, torch.bfloat16, seed=73)
        obj = b.object(A)
        want = A.attend_paged(obj, b.q, b.k, b.v)
        for _ in range(3):
            A.attend_paged(obj, -b.q, b.k, b.v)  # other pieces' results in the workspace
            obj.workspace[128:128 + 4864].view(torch.int64).fill_(1)
            assert torch.equal(A.attend_paged(obj, b.q, b.k, b.v), want)
        assert A.attn_get_status() == 0
