"""The batched kernels' second wait, that of the forms with a cap, a bias, first positions or an 8-bit cache, and those forms'
way out of a pipeline that broke, without a GPU fault (as test_batch_failure_gpu.py)."""
import pytest
import torch

from batch_ref import Batch
from cache8_ref import Batch8

pytestmark = pytest.mark.gpu


def test_the_lanes_of_a_warp_leave_a_broken_wait_together(cuda_lib):
    A = cuda_lib
    assert A.attn_get_status() == 0
    lanes = torch.full((8,), 7, dtype=torch.int32, device="cuda")
    for us in (50, 200, 1000, 3000) * 10:
        lanes.fill_(7)
        A.attn_selftest_short_wait(lanes, us)
        assert A.attn_get_status() == A.ATTN_ERR_TIMEOUT
        got = [x & 0xffffffff for x in lanes.tolist()]
        assert got[0] == 0 and all(x in (0, 0xffffffff) for x in got), got
    for bad in (0, 2000000):
        with pytest.raises(A.AttnError):
            A.attn_selftest_short_wait(lanes, bad)
    assert A.attn_get_status() == 0


def test_the_limit_holds_where_the_timers_low_word_wraps(cuda_lib):
    """It wraps every 2^32 ns: waits of 0.2 s one after the other for longer than that, none of them cut short (two
    clocks: 0.1%) or as long as two."""
    A = cuda_lib
    lanes = torch.zeros(8, dtype=torch.int32, device="cuda")
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(24)]
    marks[0].record()
    for m in marks[1:]:
        A.attn_selftest_short_wait(lanes, 200000)
        m.record()
    torch.cuda.synchronize()
    assert A.attn_get_status() == A.ATTN_ERR_TIMEOUT
    ms = [a.elapsed_time(b) for a, b in zip(marks, marks[1:])]
    assert sum(ms) > 2 ** 32 * 1e-6 and all(199.8 <= t <= 400 for t in ms), ms


@pytest.fixture
def brief_waits(cuda_lib):
    """Sets the limit of the waits inside the batched kernels; the usual one is back at the end."""
    yield cuda_lib.attn_selftest_batch_wait
    cuda_lib.attn_selftest_batch_wait(0)


SHAPES = [  # single tokens; tcgen05 on single multiprocessors and on pairs, whole and part heads
    dict(H=32, G=8, D=128, new=[1] * 20, kv=[3000] * 20),
    dict(H=14, G=2, D=64, new=[1], kv=[9000]),
    dict(H=8, G=2, D=64, new=[300, 2], kv=[4000, 900]),
    dict(H=8, G=2, D=48, new=[300, 2], kv=[4000, 900]),
    dict(H=32, G=8, D=128, new=[8, 1, 4], kv=[9000, 70, 300]),
    dict(H=10, G=2, D=96, new=[30, 4], kv=[2000, 300]),
    dict(H=32, G=8, D=128, new=[500, 256], kv=[4000, 256]),
    dict(H=8, G=8, D=80, new=[700, 600], kv=[2000, 600]),
]
FORMS = [dict(softcap=30.0), dict(alibi=True), dict(softcap=30.0, alibi=True, window=700, sinks=40),
         dict(window=700, sinks=40), dict(window=700, sinks=40, alibi=True)]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(sorted(f)))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "H%d-G%d-D%d-%d" % (c["H"], c["G"], c["D"], sum(c["new"])))
def test_calls_whose_waits_run_out_end_and_leave_later_calls_right(cuda_lib, brief_waits, shape, form, bits):
    """Each call ends, with ATTN_ERR_TIMEOUT or its usual result; the next ones, on a fresh workspace and on the same one,
    have their usual bits."""
    A, kw = cuda_lib, dict(form)
    sizes = [shape[x] for x in ("new", "kv", "H", "G", "D")]
    if kw.pop("alibi", False):
        H = shape["H"]
        kw["alibi_slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
    if bits == 8:
        b = Batch8(*sizes, 32, 16, dtype=torch.bfloat16, seed=71)
        pools, attend = (b.cache(A),), A.attend_paged8
    else:
        b = Batch(*sizes, 32, torch.bfloat16, seed=71)
        pools, attend = (b.k, b.v), A.attend_paged
    kept = b.object(A)
    want = attend(kept, b.q, *pools, **kw)
    assert A.attn_get_status() == 0
    ran_out = 0
    for ns in (1, 100, 300, 1000, 3000, 10000, 30000) * 2:
        for batch in (b.object(A), kept):
            brief_waits(ns)
            got = attend(batch, b.q, *pools, **kw)
            status = A.attn_get_status()
            brief_waits(0)
            assert status in (0, A.ATTN_ERR_TIMEOUT)
            assert status or torch.equal(got, want)
            ran_out += status != 0
            again = attend(batch, b.q, *pools, **kw)
            assert A.attn_get_status() == 0 and torch.equal(again, want)
    assert ran_out
