"""attn_batch_paged8's way out of a pipeline that broke, without a GPU fault: waits that give up within a limit, and
the calls after them (as test_batch_failure_gpu.py)."""
import pytest
import torch

from cache8_ref import Batch8

pytestmark = pytest.mark.gpu

# One batch per kernel and form: single tokens (whole and split items), tcgen05 on single multiprocessors and on pairs (Q as
# boxes and by a warp), short pieces and long ones.
BROKEN = [
    dict(H=32, G=8, D=128, new=[1] * 40, kv=[3000] * 40),
    dict(H=32, G=8, D=128, new=[1], kv=[9000]),
    dict(H=14, G=2, D=64, new=[1, 1, 1], kv=[5000, 30, 800], softcap=30.0),
    dict(H=8, G=2, D=64, new=[300, 2], kv=[4000, 900]),
    dict(H=10, G=2, D=48, new=[300, 2], kv=[4000, 900]),
    dict(H=32, G=8, D=128, new=[8, 1, 4], kv=[9000, 70, 300]),
    dict(H=12, G=4, D=96, new=[70, 1, 4], kv=[2000, 70, 300]),
    dict(H=32, G=8, D=128, new=[700, 256], kv=[4000, 256]),
    dict(H=16, G=16, D=128, new=[700, 600], kv=[2000, 600]),
    dict(H=32, G=8, D=96, new=[700, 256], kv=[4000, 256]),
]


@pytest.fixture
def brief_waits(cuda_lib):
    """Sets the limit of the waits inside the batched kernels; the usual one is back at the end."""
    yield cuda_lib.attn_selftest_batch_wait
    cuda_lib.attn_selftest_batch_wait(0)


@pytest.mark.parametrize("case", BROKEN, ids=lambda c: "H%d-G%d-D%d-%d" % (c["H"], c["G"], c["D"], sum(c["new"])))
def test_calls_whose_waits_run_out_end_and_leave_later_calls_right(cuda_lib, brief_waits, case):
    """Each call ends, with ATTN_ERR_TIMEOUT or a result; the next ones, on a fresh workspace and on the same one, have
    their usual bits."""
    A, kw = cuda_lib, dict(case)
    b = Batch8(kw.pop("new"), kw.pop("kv"), kw.pop("H"), kw.pop("G"), kw.pop("D"), 32, 16, dtype=torch.bfloat16, seed=71)
    cache, kept = b.cache(A), b.object(A)
    want = A.attend_paged8(kept, b.q, cache, **kw)
    assert A.attn_get_status() == 0
    ran_out = 0
    for ns in (1, 100, 300, 1000, 3000, 10000, 30000) * 3:
        for batch in (b.object(A), kept):
            brief_waits(ns)
            got = A.attend_paged8(batch, b.q, cache, **kw)
            status = A.attn_get_status()
            brief_waits(0)
            assert status in (0, A.ATTN_ERR_TIMEOUT)
            assert status or torch.equal(got, want)
            ran_out += status != 0
            again = A.attend_paged8(batch, b.q, cache, **kw)
            assert A.attn_get_status() == 0 and torch.equal(again, want)
    assert ran_out
