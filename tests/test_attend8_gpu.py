"""attn_batch_paged8: attention over an 8-bit paged cache, on every kernel, against a plain 64-bit form; and serving
steps of append, attention and read-back together."""
import pytest
import torch

from batch_ref import theta, turn
from cache8_ref import Batch8, attend64, tolerance

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

BATCHES = {  # new, kv, H, G, D, page_rows, scale_rows
    "tokens": ([1] * 9, [1, 2, 5, 64, 65, 300, 1000, 2049, 777], 8, 2, 64, 16, 16),
    "tokens, heads of 128": ([1] * 6, [700, 129, 4000, 17, 128, 1], 32, 8, 128, 8, 4),
    "tokens, 16 heads a kv head": ([1] * 3, [700, 2900, 17], 32, 2, 128, 64, 64),
    "tokens, heads of 96": ([1] * 4, [700, 129, 2000, 17], 14, 2, 96, 24, 3),
    "tokens, heads of 16": ([1] * 4, [70, 129, 2000, 17], 5, 5, 16, 32, 1),
    "tokens and gaps": ([1, 0, 1, 0, 1], [700, 129, 2000, 0, 40], 4, 1, 128, 40, 8),
    "more heads than a block": ([1, 1], [500, 90], 40, 2, 64, 16, 2),
    "chunks": ([3, 0, 130, 1, 64], [3, 9, 1300, 700, 64], 8, 2, 64, 16, 8),
    "chunks, heads of 48": ([40, 7], [1500, 500], 6, 3, 48, 16, 16),
    "chunks, heads of 128": ([40, 7, 90], [1500, 500, 90], 12, 4, 128, 8, 1),
    "chunks, 4 heads a kv head": ([40, 7, 33], [1500, 500, 90], 16, 4, 128, 32, 32),
    "pairs": ([300, 257], [2000, 257], 8, 2, 128, 64, 16),
    "pairs, heads of 80": ([400], [1111], 4, 2, 80, 128, 128),
    "a prompt": ([1025], [1025], 4, 1, 128, 16, 4),
    "three heads a kv head": ([200, 5], [900, 1200], 6, 2, 128, 32, 32),
    "odd pages": ([1, 70, 9], [400, 900, 9], 8, 2, 64, 7, 7),
    "odd pages, heads of 128": ([1, 1, 30], [400, 33, 500], 4, 2, 128, 5, 1),
    "small pages": ([1, 1, 50], [400, 33, 500], 4, 2, 128, 4, 2),
}


def run(A, b, q=None, **kw):
    out = torch.full_like(b.q, 7.0)
    A.attend_paged8(b.object(A), b.q if q is None else q, b.cache(A), out=out, **kw)
    assert A.attn_get_status() == 0
    assert (out[b.starts[-1]:] == 7.0).all()
    return out[:b.starts[-1]]


def check(b, out, ref, more=1.0):
    ref, mag, vmax = ref
    n = b.starts[-1]
    tol = tolerance(ref, more * mag, vmax, out.dtype, F16, max(b.kv))[:n]
    assert ((out.double() - ref[:n]).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("name", list(BATCHES))
def test_attention(cuda_lib, name, dtype):
    b = Batch8(*BATCHES[name], dtype=dtype, seed=len(name), pad=3)
    check(b, run(cuda_lib, b), attend64(b))
    wide = Batch8(*BATCHES[name], dtype=dtype, seed=1, kv_dim=b.G * b.D + 16)
    check(wide, run(cuda_lib, wide, scale=0.3), attend64(wide, scale=0.3), 4.0)  # (scores three times as large)


@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 0), (100, 3), (33, 130), (500, 40)])
@pytest.mark.parametrize("name", list(BATCHES))
def test_window_and_sinks(cuda_lib, name, window, sinks):
    b = Batch8(*BATCHES[name], dtype=F16, seed=window)
    check(b, run(cuda_lib, b, window=window, sinks=sinks), attend64(b, window=window, sinks=sinks))


@pytest.mark.parametrize("name", ["tokens", "tokens, heads of 128", "chunks", "chunks, heads of 128", "pairs", "odd pages"])
@pytest.mark.parametrize("how", [dict(softcap=20.0), dict(alibi=True), dict(prefix=True), dict(scale=-0.1),
                                 dict(softcap=1.5, alibi=True, prefix=True, window=90, sinks=20)])
def test_caps_biases_and_prefixes(cuda_lib, name, how):
    b = Batch8(*BATCHES[name], dtype=BF16, seed=3)
    H = b.H
    slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=F32) / H) if how.get("alibi") else None
    prefix = [n * 2 // 3 for n in b.kv] if how.get("prefix") else None
    kw = {k: v for k, v in how.items() if k not in ("alibi", "prefix")}
    out = run(cuda_lib, b, alibi_slopes=slopes, prefix_len=b.dev(prefix) if prefix else None, **kw)
    # The bias is off by 2^-24 of up to 2048: another 2^-13 of a weight.
    check(b, out, attend64(b, slopes=slopes, prefix=prefix, **kw), 2.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("name", ["tokens, heads of 128", "chunks", "pairs", "odd pages"])
def test_rows_of_any_size(cuda_lib, name, dtype):
    """Q from 2^-90 to 2^90 (bf16) with the scale that undoes it, small entries beside large ones, rows of zeros."""
    A = cuda_lib
    b = Batch8(*BATCHES[name], dtype=dtype, seed=5)
    for p in ((-90, -20, 90) if dtype == BF16 else (-4, 4)):
        q = b.q.double() * 2.0 ** p
        q[:, ::3] *= 2.0 ** -7
        q[0] = 0
        q = q.to(dtype)
        scale = 2.0 ** -p / 8
        check(b, run(A, b, q=q, scale=scale), attend64(b, q=q, scale=scale), 2.0)


@pytest.mark.parametrize("name", list(BATCHES))
def test_hidden_positions_do_not_show(cuda_lib, name):
    """NaN codes and any scale at positions that no row attends."""
    A = cuda_lib
    window, sinks = 40, 5
    new, kv, _, _, D, _, sr = BATCHES[name]
    b = Batch8(*BATCHES[name], dtype=BF16, seed=4)
    want = run(A, b, window=window, sinks=sinks)
    for i, (n, length) in enumerate(zip(new, kv)):
        lo = max(0, length - n + 1 - window)
        if n and lo > sinks:
            sl = b.slots(i, sinks, lo)
            for x in "kv":
                b.codes[x][sl] = 0xff
            first = (sinks + sr - 1) // sr * sr
            whole = b.slots(i, first, max(first, lo // sr * sr))  # blocks that hold no other position
            for x in "kv":
                b.scales[x][whole // sr] = 255
    assert torch.equal(want, run(A, b, window=window, sinks=sinks))


@pytest.mark.parametrize("name", ["tokens", "chunks, heads of 128", "pairs"])
def test_scales_at_the_ends_of_their_range(cuda_lib, name):
    """Scales of 2^-14 and 2^7, and bytes outside, which read as these."""
    A = cuda_lib
    b = Batch8(*BATCHES[name], dtype=BF16, seed=6)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x, choice in (("k", [0, 113, 114, 116]), ("v", [0, 113, 120, 134, 255])):
        pick = torch.randint(0, len(choice), b.scales[x].shape, generator=g, device="cuda")
        b.scales[x] = torch.tensor(choice, dtype=torch.uint8, device="cuda")[pick]
    ok = ~(b.k.isnan())
    b.k, b.v = (torch.where(ok, b.values(x), float("nan")) for x in "kv")
    check(b, run(A, b, scale=8.0), attend64(b, scale=8.0), 2.0)


def test_splits_graphs_streams_and_repeated_calls(cuda_lib):
    A = cuda_lib
    for new, H, D in (([4, 1], 16, 128), ([1, 1], 8, 64), ([1, 1], 32, 128), ([700, 600], 8, 128)):
        b = Batch8(new, [60000, 30001], H, 2, D, 64, 16, dtype=BF16, seed=6)
        batch, cache = b.object(A), b.cache(A)
        want = A.attend_paged8(batch, b.q, cache, window=9000, sinks=700)
        out = torch.empty_like(b.q)
        for _ in range(3):
            assert torch.equal(want, A.attend_paged8(batch, b.q, cache, window=9000, sinks=700, out=out))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = A.attend_paged8(batch, b.q, cache, window=9000, sinks=700, stream=side)
        side.synchronize()
        assert torch.equal(want, got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            A.attend_paged8(batch, b.q, cache, out=out, window=9000, sinks=700)
        for kv in ([60000, 30001], [9702, 701], [20000, 700]):
            b.kv = kv
            b.kv_len.copy_(b.dev(kv))
            graph.replay()
            assert A.attn_get_status() == 0
            check(b, out, attend64(b, window=9000, sinks=700))


def test_a_workspace_serves_both_caches(cuda_lib):
    """Calls of one batch object over 16-bit and 8-bit pools, in turn."""
    A = cuda_lib
    b = Batch8([1, 300], [5000, 900], 8, 2, 128, 16, 16, dtype=F16, seed=7)
    batch, cache = b.object(A), b.cache(A)
    eight, sixteen = A.attend_paged8(batch, b.q, cache), A.attend_paged(batch, b.q, b.k, b.v)
    for _ in range(3):
        assert torch.equal(eight, A.attend_paged8(batch, b.q, cache))
        assert torch.equal(sixteen, A.attend_paged(batch, b.q, b.k, b.v))
    check(b, eight, attend64(b))


def test_bad_device_values(cuda_lib):
    """A page outside the pool reads as zeros, and is reported."""
    A = cuda_lib
    for new, D in (([1, 1], 128), ([9, 3], 128), ([300, 300], 128), ([9, 3], 64)):
        b = Batch8(new, [400, 333], 4, 2, D, 16, 16, dtype=BF16, seed=8)
        table = b.block_table.clone()
        table[0, 3] = b.num_pages
        A.attend_paged8(b.object(A, block_table=table), b.q, b.cache(A))
        assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
        sl = b.slots(0, 48, 64)
        b.k[sl], b.v[sl] = 0, 0
        got = A.attend_paged8(b.object(A, block_table=table), b.q, b.cache(A))
        assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
        check(b, got, attend64(b))


@pytest.mark.parametrize("src,H,G,D,page_rows,scale_rows", [(BF16, 32, 8, 128, 16, 16), (F32, 6, 2, 64, 24, 8),
                                                           (F16, 4, 4, 96, 32, 1), (BF16, 4, 2, 128, 7, 7)])
def test_serving_steps(cuda_lib, src, H, G, D, page_rows, scale_rows):
    """Prompts, then tokens: head norms, rotary turn and append, attention with window and sinks over what the cache
    holds, and the cache read back; each step against 64 bits from the values that the cache then holds."""
    A = cuda_lib
    new, window, sinks = [90, 1, 40], 50, 4
    b = Batch8(new, [200, 200, 200], H, G, D, page_rows, scale_rows, dtype=BF16 if src == F32 else src, seed=9)
    b.kv = list(new)
    batch, cache = b.object(A), b.cache(A)
    g = torch.Generator(device="cuda").manual_seed(10)
    mk = lambda n, h: torch.randn(n, h * D, generator=g, device="cuda").to(src)  # noqa: E731
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda").to(src) for _ in range(2))
    table, th = A.rope_table(256, D), theta(D)
    for step in range(5):
        starts = [sum(b.new[:i]) for i in range(4)]
        b.starts, b.rows = starts, starts[-1]
        batch.q_start.copy_(b.dev(starts))
        batch.kv_len.copy_(b.dev(b.kv))
        q, k, v = mk(b.rows, H), mk(b.rows, G), mk(b.rows, G)
        qt = A.append_paged8(batch, k, v, cache, q=q, table=table, q_weight=wq, k_weight=wk)
        out = A.attend_paged8(batch, qt, cache, window=window, sinks=sinks)
        rows = sum(b.kv)
        ks, vs = (torch.empty(rows, G * D, dtype=b.dtype, device="cuda") for _ in range(2))
        A.read_paged8(batch, cache, b.dev([sum(b.kv[:i]) for i in range(4)]), ks, vs)
        assert A.attn_get_status() == 0
        sl = torch.cat([b.slots(i, 0, n) for i, n in enumerate(b.kv)])
        assert torch.equal(ks.double(), b.values("k")[sl]) and torch.equal(vs.double(), b.values("v")[sl])
        b.k, b.v = b.values("k"), b.values("v")
        check(b, out, attend64(b, q=qt, window=window, sinks=sinks), 2.0)  # (normed heads: larger scores)
        # The step's K within the steps of its codes: half a step is 2^-4 of a value, and one of 2^-10 of the block's
        # scale, which is below 2^-7 of its largest value.
        pos = torch.cat([torch.arange(n - m, n) for m, n in zip(b.new, b.kv)]).cuda()
        x = k.double().view(-1, G, D)
        x = turn(x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wk.double(), pos, th, False).view(b.rows, -1)
        at = torch.cat([b.slots(i, n - m, n) for i, (m, n) in enumerate(zip(b.new, b.kv))])
        assert ((b.k[at, :G * D] - x).abs() <= 1.01 * 2.0 ** -4 * x.abs() + 2.0 ** -17 * x.abs().max()).all()
        b.new = [1, 1, 1] if step else [1, 30, 0]
        b.kv = [n + m for n, m in zip(b.kv, b.new)]


def test_refusals(cuda_lib):
    A = cuda_lib
    b = Batch8([1], [5], 2, 1, 64, 8, 8)
    batch, cache = b.object(A), b.cache(A)
    for bad in (dict(sinks=-1, window=4), dict(window=2 ** 32), dict(out=torch.empty_like(b.q).half()),
                dict(alibi_slopes=torch.ones(3, device="cuda")), dict(prefix_len=b.dev([1, 2]))):
        with pytest.raises(ValueError):
            A.attend_paged8(batch, b.q, cache, **bad)
    with pytest.raises(A.AttnError):
        A.attend_paged8(batch, b.q.float(), cache)
    other = Batch8([1], [5], 2, 1, 64, 12, 4)
    with pytest.raises(ValueError, match="fit the batch"):
        A.attend_paged8(batch, b.q, A.PagedCache8(*(torch.zeros(s, dtype=torch.uint8, device="cuda")
                                                    for s in ((32, 64), (32, 64), (2, 2), (2, 2)))))
    with pytest.raises(ValueError, match="fit the batch"):
        A.append_paged8(batch, b.q[:, :64], b.q[:, :64], other.cache(A))
    with pytest.raises(AttributeError):
        cache.scale_rows = 4


def test_blocks_of_a_pair_read_each_others_latest_operands(cuda_lib):
    """Each block of a pair makes half of every operand tile and the first one multiplies all of them: with other codes in
    the same pages at every replay, results are those of the codes of that replay."""
    A = cuda_lib
    b = Batch8([512, 300], [3000, 2100], 8, 2, 128, 64, 16, dtype=BF16, seed=12)
    batch, cache = b.object(A), b.cache(A)
    out = torch.empty_like(b.q)
    graph = torch.cuda.CUDAGraph()
    A.attend_paged8(batch, b.q, cache, out=out)
    with torch.cuda.graph(graph):
        A.attend_paged8(batch, b.q, cache, out=out)
    g = torch.Generator(device="cuda").manual_seed(13)
    codes = {x: b.codes[x].clone() for x in "kv"}
    for step in range(40):
        flip = torch.randint(0, 2, (2, b.codes["k"].shape[0], 1), generator=g, device="cuda", dtype=torch.uint8) * 0x80
        for x, f in zip("kv", flip):  # other signs of whole rows
            b.codes[x].copy_(codes[x] ^ f)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, A.attend_paged8(batch, b.q, cache)) and A.attn_get_status() == 0
        if step % 10 == 0:
            own = ~b.k.isnan()
            b.k, b.v = (torch.where(own, b.values(x).to(BF16), float("nan")) for x in "kv")
            check(b, got, attend64(b))
