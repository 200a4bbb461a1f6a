"""attn_batch_paged_sinks: a sliding window with first positions that stay visible, on every kernel of the batched
attention, against a plain 64-bit form."""
import pytest
import torch

from batch_ref import Batch
from cache8_ref import attend64, tolerance

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16

BATCHES = {  # new, kv, H, G, D, page_rows
    "tokens": ([1] * 9, [1, 2, 5, 64, 65, 300, 1000, 2049, 777], 8, 2, 64, 16),
    "tokens, heads of 128": ([1] * 5, [700, 129, 4000, 17, 128], 32, 8, 128, 8),
    "tokens, heads of 96": ([1] * 4, [700, 129, 2000, 17], 14, 2, 96, 24),
    "chunks": ([3, 0, 130, 1, 64], [3, 9, 1300, 700, 64], 8, 2, 64, 16),
    "chunks, heads of 128": ([40, 7, 90], [1500, 500, 90], 12, 4, 128, 8),
    "pairs": ([300, 257], [2000, 257], 8, 2, 128, 64),
    "pairs, heads of 80": ([400], [1111], 4, 2, 80, 128),
    "three heads a kv head": ([200, 5], [900, 1200], 6, 2, 128, 32),
    "odd pages": ([1, 70, 9], [400, 900, 9], 8, 2, 64, 7),
    "odd pages, heads of 128": ([1, 1, 30], [400, 33, 500], 4, 2, 128, 5),
}


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (100, 3), (64, 64), (33, 130), (500, 40), (200, 2 ** 32 - 1)])
@pytest.mark.parametrize("name", list(BATCHES))
def test_window_and_sinks(cuda_lib, name, window, sinks, dtype):
    A = cuda_lib
    new, kv, H, G, D, pr = BATCHES[name]
    b = Batch(new, kv, H, G, D, pr, dtype, seed=window, pad=3)
    out = torch.full_like(b.q, 7.0)
    A.attend_paged(b.object(A), b.q, b.k, b.v, out=out, window=window, sinks=sinks)
    assert A.attn_get_status() == 0
    ref, mag, vmax = attend64(b, window=window, sinks=sinks)
    n = b.starts[-1]
    assert ((out[:n].double() - ref[:n]).abs() <= tolerance(ref, mag, vmax, dtype, dtype, max(kv))[:n]).all()
    assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("name", ["tokens", "chunks, heads of 128", "pairs", "odd pages"])
@pytest.mark.parametrize("how", [dict(softcap=20.0), dict(alibi=True), dict(prefix=True), dict(softcap=5.0, alibi=True, prefix=True),
                                 dict(scale=-0.1)])
def test_with_caps_biases_and_prefixes(cuda_lib, name, how):
    A = cuda_lib
    new, kv, H, G, D, pr = BATCHES[name]
    b = Batch(new, kv, H, G, D, pr, F16, seed=3)
    slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H) if how.get("alibi") else None
    prefix = [n * 2 // 3 for n in kv] if how.get("prefix") else None
    kw = dict(window=90, sinks=20, softcap=how.get("softcap", 0.0), scale=how.get("scale"))
    out = A.attend_paged(b.object(A), b.q, b.k, b.v, alibi_slopes=slopes, prefix_len=b.dev(prefix) if prefix else None,
                         **kw)
    assert A.attn_get_status() == 0
    ref, mag, vmax = attend64(b, slopes=slopes, prefix=prefix, **kw)
    # The bias is a product of up to 2048 * 2^-1 in fp32, off by 2^-24 of it: another 2^-14 of a weight, at most 2^-12 of all.
    assert ((out.double() - ref).abs() <= tolerance(ref, 2 * mag, vmax, F16, F16, max(kv))).all()


@pytest.mark.parametrize("name", list(BATCHES))
def test_hidden_positions_do_not_show(cuda_lib, name):
    """NaN and infinities at positions that no row attends, beside the first ones and before the window."""
    A = cuda_lib
    new, kv, H, G, D, pr = BATCHES[name]
    window, sinks = 40, 5
    b = Batch(new, kv, H, G, D, pr, BF16, seed=4)
    want = A.attend_paged(b.object(A), b.q, b.k, b.v, window=window, sinks=sinks)
    for i, (n, length) in enumerate(zip(new, kv)):
        lo = max(0, length - n + 1 - window)
        if n and lo > sinks:
            sl = b.slots(i, sinks, lo)
            b.k[sl], b.v[sl] = float("nan"), float("inf")
    got = A.attend_paged(b.object(A), b.q, b.k, b.v, window=window, sinks=sinks)
    assert A.attn_get_status() == 0 and torch.equal(want, got)


@pytest.mark.parametrize("name", ["tokens", "chunks", "pairs", "odd pages"])
def test_without_effect_it_is_the_plain_call(cuda_lib, name):
    """No window, no sinks, or a window as long as the sequences: the same bits as without."""
    A = cuda_lib
    new, kv, H, G, D, pr = BATCHES[name]
    b = Batch(new, kv, H, G, D, pr, F16, seed=5)
    batch = b.object(A)
    plain = A.attend_paged(batch, b.q, b.k, b.v)
    assert torch.equal(plain, A.attend_paged(batch, b.q, b.k, b.v, sinks=10))
    assert torch.equal(plain, A.attend_paged(batch, b.q, b.k, b.v, window=max(kv), sinks=3))
    windowed = A.attend_paged(batch, b.q, b.k, b.v, window=50)
    assert torch.equal(windowed, A.attend_paged(batch, b.q, b.k, b.v, window=50, sinks=0))
    assert torch.equal(windowed, A.attend_paged(batch, b.q, b.k, b.v, window=50))


def test_a_long_cache_reads_its_ends_alone(cuda_lib):
    """Split keys: pieces that hold first positions and window, in a captured graph as lengths grow."""
    A = cuda_lib
    b = Batch([4, 1], [60000, 30001], 16, 2, 128, 64, BF16, seed=6, junk=0.0)
    batch = b.object(A)
    out = torch.empty_like(b.q)
    A.attend_paged(batch, b.q, b.k, b.v, out=out, window=9000, sinks=700)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        A.attend_paged(batch, b.q, b.k, b.v, out=out, window=9000, sinks=700)
    for kv in ([60000, 30001], [9702, 701], [20000, 4]):
        b.kv = kv
        b.kv_len.copy_(b.dev(kv))
        graph.replay()
        assert A.attn_get_status() == 0
        ref, mag, vmax = attend64(b, window=9000, sinks=700)
        assert ((out.double() - ref).abs() <= tolerance(ref, mag, vmax, BF16, BF16, max(kv))).all()


def test_refusals(cuda_lib):
    A = cuda_lib
    b = Batch([1], [5], 2, 1, 64, 8, BF16)
    for bad in (dict(sinks=-1, window=4), dict(sinks=2 ** 32, window=4)):
        with pytest.raises(ValueError, match="sinks"):
            A.attend_paged(b.object(A), b.q, b.k, b.v, **bad)
