"""attn_batch_paged (attention of a ragged batch's new tokens over a paged
16-bit cache) against a plain 64-bit form.

Pools are shuffled pages; every pool row that no sequence owns holds NaN, so
reading past a sequence or through a wrong page shows."""
import pytest
import torch

from batch_ref import Batch, attend_tolerance

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
CUT = float("nan")


def check(A, b, where="", q=None, **kw):
    rows = b.starts[-1]
    keep = torch.full((b.rows, b.H * b.D), 7.0, dtype=b.dtype, device="cuda")
    call = dict(kw)
    if "prefix" in call:
        call["prefix_len"] = b.dev(call.pop("prefix"))
    if "slopes" in call:
        call["alibi_slopes"] = call.pop("slopes")
    got = A.attend_paged(b.object(A), b.q if q is None else q, b.k, b.v, out=keep, **call)
    torch.cuda.synchronize()
    assert A.attn_get_status() == 0
    ref, mag = b.attend(q=q, **kw)
    err = (got[:rows].double() - ref[:rows]).abs()
    assert torch.isfinite(got[:rows].float()).all(), where + ": non-finite output"
    tol = attend_tolerance(ref, mag, b.dtype, max(b.kv + [1]))[:rows]
    bad = err > tol
    assert not bad.any(), "%s: %d of %d off, worst err/tol %.3g" % (where, int(bad.sum()), bad.numel(),
                                                                    float((err / tol).max()))
    assert (got[rows:] == 7.0).all(), where + ": rows of no sequence were written"
    return got


HEADS = [(1, 1, 64), (8, 2, 64), (32, 8, 128), (7, 1, 128), (16, 16, 64), (20, 4, 128), (16, 1, 64), (6, 2, 80),
         (5, 5, 8), (10, 2, 120), (4, 2, 96), (130, 1, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,G,D", HEADS)
def test_single_tokens(cuda_lib, H, G, D, dtype):
    """One new token a sequence; lengths around tile, page and split borders."""
    kv = [1, 2, 63, 64, 65, 127, 128, 129, 257, 1000]
    check(cuda_lib, Batch([1] * len(kv), kv, H, G, D, 32, dtype, seed=H), "decode H%d G%d D%d" % (H, G, D))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,G,D", HEADS)
def test_chunks(cuda_lib, H, G, D, dtype):
    """Prompts, chunks behind a cache and single tokens in one batch, an empty sequence among them."""
    new = [5, 0, 1, 64, 130, 33, 1]
    kv = [5, 40, 300, 64, 511, 129, 1]
    check(cuda_lib, Batch(new, kv, H, G, D, 16, dtype, seed=H + 1, pad=3), "chunks H%d G%d D%d" % (H, G, D))


@pytest.mark.parametrize("page_rows", [1, 7, 8, 16, 24, 48, 64, 100, 128, 256, 512])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(cuda_lib, page_rows, D):
    b = Batch([1, 70, 200], [333, 70, 700], 8, 2, D, page_rows, BF16, seed=page_rows)
    check(cuda_lib, b, "page_rows %d" % page_rows)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 128, 1000, 2 ** 32 - 1])
def test_window(cuda_lib, window, dtype):
    """Pages before a window hold NaN: they must not be read into a result."""
    b = Batch([1, 1, 90, 150], [50, 700, 90, 900], 8, 2, 64, 16, dtype, seed=window % 97)
    if window < 2 ** 31:
        for i, (n, length) in enumerate(zip(b.new, b.kv)):
            gone = max(0, length - n + 1 - window)
            if gone:
                sl = b.slots(i, 0, gone)
                b.k[sl] = CUT
                b.v[sl] = CUT
    check(cuda_lib, b, "window %d" % window, window=window if window < 2 ** 31 else 0)
    if window >= 2 ** 31:
        got = cuda_lib.attend_paged(b.object(cuda_lib), b.q, b.k, b.v, window=window)
        assert torch.equal(got, cuda_lib.attend_paged(b.object(cuda_lib), b.q, b.k, b.v))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [1.0, 30.0, 50.0, 1e4])
def test_softcap(cuda_lib, softcap, D, dtype):
    b = Batch([1, 1, 77, 140], [600, 17, 77, 400], 14, 2, D, 32, dtype, seed=3)
    check(cuda_lib, b, "cap %g" % softcap, softcap=softcap)


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_distance_bias(cuda_lib, softcap, prefix):
    b = Batch([1, 1, 77, 140], [600, 17, 77, 400], 16, 4, 128, 64, BF16, seed=4)
    slopes = 2.0 ** (-0.5 * torch.arange(1, 17, device="cuda", dtype=torch.float32))
    kw = dict(prefix=[100, 17, 30, 399]) if prefix else {}
    check(cuda_lib, b, "alibi", slopes=slopes, softcap=softcap, **kw)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("prefix", [[0, 0, 0, 0], [1, 5, 64, 128], [600, 17, 77, 400], [300, 2, 40, 261]])
def test_prefix(cuda_lib, prefix, window):
    """Keys below the prefix are visible to every row (a prefix longer than the sequence is cut)."""
    b = Batch([1, 3, 77, 140], [600, 17, 77, 400], 8, 2, 64, 16, F16, seed=5)
    check(cuda_lib, b, "prefix", prefix=prefix, window=window)


def test_prefix_past_the_sequence_is_cut(cuda_lib):
    b = Batch([3, 9], [30, 9], 4, 2, 64, 16, BF16, seed=6)
    A, obj = cuda_lib, b.object(cuda_lib)
    got = A.attend_paged(obj, b.q, b.k, b.v, prefix_len=b.dev([2 ** 31 - 1, 10]))
    want = A.attend_paged(obj, b.q, b.k, b.v, prefix_len=b.dev([30, 9]))
    torch.cuda.synchronize()
    assert A.attn_get_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("H,G,D,new,kv", [
    (32, 8, 128, [1], [20000]),            # few rows, many keys: split over the GPU
    (8, 8, 64, [1] * 3, [30000, 1, 5]),
    (32, 8, 128, [200], [9000]),
    (8, 1, 128, [1] * 150, list(range(1, 3000, 20))),
    (4, 4, 128, [900, 1, 300], [900, 4000, 2300]),
])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_split_items(cuda_lib, H, G, D, new, kv, dtype):
    check(cuda_lib, Batch(new, kv, H, G, D, 64, dtype, seed=7), "split")


def test_large_scores(cuda_lib):
    """Scores of standard deviation 30 (near one-hot rows), exact ties and a constant cache.  The score error
    allowed for in the tolerance grows with the scores: 128 * 2^-24 * (16 * 30) < 2^-8, twice that in a weight."""
    b = Batch([1, 40], [500, 300], 8, 2, 128, 32, BF16, seed=8)
    q = (b.q.float() * 30).to(BF16)
    got = cuda_lib.attend_paged(b.object(cuda_lib), q, b.k, b.v)
    ref, mag = b.attend(q=q)
    tol = attend_tolerance(ref, mag, BF16, 500) + 2.0 ** -7 * mag
    assert ((got.double() - ref).abs() <= tol).all()
    for i, n in enumerate(b.kv):
        b.k[b.slots(i, 0, n)] = 0.5
    check(cuda_lib, b, "ties")


def test_repeated_calls_give_identical_bits_and_graph_replays_as_lengths_grow(cuda_lib):
    A = cuda_lib
    kv = [9, 700, 64, 2000]
    b = Batch([1] * 4, kv, 32, 8, 128, 16, BF16, seed=9)
    obj = b.object(A)
    out = torch.zeros_like(b.q)
    first = A.attend_paged(obj, b.q, b.k, b.v).clone()
    for _ in range(3):
        assert torch.equal(first, A.attend_paged(obj, b.q, b.k, b.v, out=out))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        A.attend_paged(obj, b.q, b.k, b.v, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.attend_paged(obj, b.q, b.k, b.v, out=out)
    for lens in ([1, 1, 1, 1], kv, [5, 300, 1, 1999]):
        b.kv_len.copy_(b.dev(lens))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        b.kv = lens
        ref, mag = b.attend()
        assert ((out.double() - ref).abs() <= attend_tolerance(ref, mag, BF16, 2000)).all()
    assert A.attn_get_status() == 0


def test_strided_rows_wide_pools_and_another_stream(cuda_lib):
    A = cuda_lib
    b = Batch([1, 100], [400, 250], 8, 2, 64, 32, BF16, seed=10, kv_dim=192)
    ref, mag = b.attend()
    wide_q = torch.full((b.rows, 8 * 64 + 40), float("nan"), dtype=BF16, device="cuda")
    wide_q[:, :512] = b.q
    wide_o = torch.full((b.rows, 8 * 64 + 8), 3.0, dtype=BF16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    A.attend_paged(b.object(A), wide_q[:, :512], b.k, b.v, out=wide_o[:, :512], stream=stream)
    torch.cuda.synchronize()
    assert ((wide_o[:, :512].double() - ref).abs() <= attend_tolerance(ref, mag, BF16, 400)).all()
    assert (wide_o[:, 512:] == 3.0).all()


def test_bad_device_values_are_reported_and_stay_in_bounds(cuda_lib):
    """Values only the device sees: a page outside the pool reads as zeros, a length past the capacity is cut, a
    length below the new rows leaves rows empty, a descending q_start leaves the sequence out."""
    A = cuda_lib
    b = Batch([1, 4, 2], [40, 60, 33], 4, 2, 64, 16, BF16, seed=11, extra_blocks=0)
    table = b.table.clone()
    bad = torch.tensor([[0, 1, -1, 2], [0, 1, 2, 3], [1, 2, 3, 4]], dtype=torch.int32)
    table[:, :4] = torch.where(bad == -1, torch.full_like(bad, 2 ** 31 - 1), bad)
    b.k.zero_()
    b.v.fill_(1.0)
    out = A.attend_paged(b.object(A, block_table=table.cuda()), b.q, b.k, b.v)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    # Equal scores: sequence 0 averages 32 ones and the 8 zeros of positions 32..39.
    assert torch.allclose(out[0].float(), torch.full((256,), 32 / 40, device="cuda"), atol=2 ** -8)
    assert torch.allclose(out[1:].float(), torch.ones(6, 256, device="cuda"))
    good = b.block_table
    out = A.attend_paged(b.object(A, kv_len=b.dev([40, 2, 10 ** 6])), b.q, b.k, b.v)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    assert (out[1:3] == 0).all() and torch.isfinite(out.float()).all()
    assert good.shape[1] == 4
    out = A.attend_paged(b.object(A, q_start=b.dev([0, 1, 0, 7])), b.q, b.k, b.v)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    out = A.attend_paged(b.object(A, q_start=b.dev([0, 1, 5, 2 ** 31 - 1])), b.q, b.k, b.v)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    assert (out[5:] == 0).all()


def test_rows_without_keys_write_zeros(cuda_lib):
    A = cuda_lib
    b = Batch([2, 3], [64, 64], 8, 2, 128, 32, F16, seed=12)
    out = torch.full_like(b.q, 5.0)
    A.attend_paged(b.object(A, kv_len=b.dev([64, 0])), b.q, b.k, b.v, out=out)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    assert (out[2:] == 0).all() and torch.isfinite(out.float()).all()


def test_many_short_sequences(cuda_lib):
    n = 3000
    kv = [1 + (i * 7) % 40 for i in range(n)]
    check(cuda_lib, Batch([1] * n, kv, 4, 2, 64, 16, BF16, seed=13), "3000 sequences")


def test_refused_workspace_and_types(cuda_lib):
    A = cuda_lib
    b = Batch([1], [20], 4, 2, 64, 16, BF16, seed=14)
    obj = b.object(A)
    obj.workspace = obj.workspace[:-1]
    out = torch.full_like(b.q, 9.0)
    with pytest.raises(A.AttnError):
        A.attend_paged(obj, b.q, b.k, b.v, out=out)
    obj = b.object(A)
    with pytest.raises(ValueError):
        A.attend_paged(obj, b.q, b.k.half(), b.v, out=out)
    with pytest.raises(A.AttnError):
        A.attend_paged(obj, b.q.float(), b.k.float(), b.v.float())
    with pytest.raises(ValueError):
        A.attend_paged(obj, b.q, b.k[:-1], b.v[:-1], out=out)
    with pytest.raises(ValueError):
        A.attend_paged(obj, b.q, b.k, b.v, out=out, prefix_len=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        A.attend_paged(obj, b.q, b.k.cpu(), b.v.cpu(), out=out)
    torch.cuda.synchronize()
    assert (out == 9.0).all()


LONG = dict(new=[700, 1, 513, 0, 256, 255, 40], kv=[700, 2000, 900, 77, 300, 4000, 131])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,G,page_rows", [(4, 4, 64), (8, 2, 16), (32, 8, 128), (8, 1, 8), (16, 1, 24), (128, 1, 32),
                                           (3, 1, 64), (10, 2, 64)])
def test_many_rows(cuda_lib, H, G, page_rows, dtype):
    """Batches of mostly long chunks, at head dimension 128 and 64."""
    for D in (128, 64):
        b = Batch(LONG["new"], LONG["kv"], H, G, D, page_rows, dtype, seed=H + page_rows, pad=2)
        check(cuda_lib, b, "long chunks H%d G%d D%d" % (H, G, D))


@pytest.mark.parametrize("kw", [
    dict(softcap=30.0), dict(window=1), dict(window=200), dict(window=1000, softcap=5.0), dict(prefix=True),
    dict(slopes=True), dict(slopes=True, prefix=True, window=300, softcap=50.0), dict(scale=0.0), dict(scale=-0.1)])
def test_many_rows_with_masks_and_maps(cuda_lib, kw):
    b = Batch(LONG["new"], LONG["kv"], 16, 4, 128, 16, BF16, seed=21)
    kw = dict(kw)
    if kw.get("prefix"):
        kw["prefix"] = [350, 2000, 1, 77, 44, 3900, 131]
    if kw.get("slopes"):
        kw["slopes"] = 2.0 ** (-0.5 * torch.arange(1, 17, device="cuda", dtype=torch.float32))
    if kw.get("window") and "prefix" not in kw:
        for i, (n, length) in enumerate(zip(b.new, b.kv)):
            gone = max(0, length - n + 1 - kw["window"])
            if gone:
                sl = b.slots(i, 0, gone)
                b.k[sl] = CUT
                b.v[sl] = CUT
    check(cuda_lib, b, str(kw), **kw)


@pytest.mark.parametrize("H,G,D,page_rows,dtype", [(8, 2, 8, 16, F16), (6, 2, 40, 64, BF16), (8, 4, 56, 8, F16),
                                                   (8, 2, 72, 64, BF16), (16, 4, 96, 16, F16), (5, 1, 96, 32, BF16),
                                                   (128, 1, 120, 64, F16), (40, 8, 80, 128, BF16)])
def test_many_rows_other_head_dims(cuda_lib, H, G, D, page_rows, dtype):
    """Head dimensions between the tile widths, chunks and single tokens; NaN between the rows of the pools."""
    for new, kv in ((LONG["new"], LONG["kv"]), ([1, 0, 1, 1, 1], [2500, 9, 1, 700, 65])):
        b = Batch(new, kv, H, G, D, page_rows, dtype, seed=H + D, pad=2, kv_dim=G * D + 16)
        b.k[:, G * D:] = float("nan")
        b.v[:, G * D:] = float("nan")
        check(cuda_lib, b, "H%d G%d D%d" % (H, G, D))
        if D > 64:
            check(cuda_lib, b, "capped", softcap=20.0, window=150)


@pytest.mark.parametrize("H,G,D,dtype", [(32, 8, 128, BF16), (14, 2, 64, F16), (12, 4, 96, BF16)])
@pytest.mark.parametrize("new,kv", [([4], [16000]), ([8], [9000]), ([9], [9000]), ([2, 0, 3, 1], [5000, 7, 6001, 130]),
                                    ([33, 2], [700, 12000])])
def test_few_rows_over_many_splits(cuda_lib, H, G, D, dtype, new, kv):
    """A few tokens behind long caches: items of few rows cut into many pieces, joined by several warps."""
    b = Batch(new, kv, H, G, D, 32, dtype, seed=51, pad=1)
    check(cuda_lib, b, "few rows H%d G%d D%d" % (H, G, D))
    obj = b.object(cuda_lib)
    first = cuda_lib.attend_paged(obj, b.q, b.k, b.v)
    for _ in range(5):
        assert torch.equal(first, cuda_lib.attend_paged(obj, b.q, b.k, b.v))


def test_many_rows_repeat_bits(cuda_lib):
    b = Batch(LONG["new"], LONG["kv"], 32, 8, 128, 64, BF16, seed=22)
    obj = b.object(cuda_lib)
    first = cuda_lib.attend_paged(obj, b.q, b.k, b.v)
    for _ in range(20):
        assert torch.equal(first, cuda_lib.attend_paged(obj, b.q, b.k, b.v))


DECODE_KV = [1, 2, 63, 64, 65, 127, 128, 129, 300, 1000, 4097, 9000]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [
    dict(), dict(window=1), dict(window=65), dict(window=1000), dict(softcap=2.0), dict(softcap=50.0, window=3000),
    dict(slopes=True), dict(slopes=True, softcap=20.0), dict(prefix=True, window=100), dict(scale=-0.05), dict(scale=0.0)])
def test_single_tokens_with_masks_and_maps(cuda_lib, kw, D):
    kw = dict(kw)
    b = Batch([1] * len(DECODE_KV), DECODE_KV, 12, 2, D, 16, F16 if D == 64 else BF16, seed=31)
    if kw.get("slopes"):
        kw["slopes"] = 2.0 ** (-0.7 * torch.arange(1, 13, device="cuda", dtype=torch.float32))
    if kw.get("prefix"):
        kw["prefix"] = [1, 1, 63, 5, 65, 100, 0, 129, 150, 1000, 4000, 2]
    elif kw.get("window"):
        for i, n in enumerate(b.kv):
            gone = max(0, n - kw["window"])
            if gone:
                sl = b.slots(i, 0, gone)
                b.k[sl] = CUT
                b.v[sl] = CUT
    check(cuda_lib, b, str(kw), **kw)


@pytest.mark.parametrize("page_rows", [8, 16, 24, 64, 100, 128, 256])
@pytest.mark.parametrize("H,G,D", [(8, 8, 128), (32, 2, 64), (15, 3, 128)])
def test_single_tokens_page_sizes(cuda_lib, H, G, D, page_rows):
    check(cuda_lib, Batch([1, 0, 1, 1], [700, 5, 41, 2500], H, G, D, page_rows, BF16, seed=page_rows), "pages")


@pytest.mark.parametrize("H,G,D,kv", [(32, 8, 128, [16384]), (8, 1, 128, [40000, 3, 700]), (16, 2, 64, [20000] * 5),
                                      (32, 8, 128, [3000] * 40)])
def test_single_tokens_repeat_bits_and_share_a_workspace(cuda_lib, H, G, D, kv):
    """Fifty calls give the same bits, also between calls of other sizes on the same workspace."""
    A = cuda_lib
    b = Batch([1] * len(kv), kv, H, G, D, 64, BF16, seed=33)
    other = Batch([300, 20], [5000, 20], H, G, D, 64, BF16, seed=34)
    obj, obj2 = b.object(A), other.object(A)
    obj2.workspace = obj.workspace
    first = check(A, b, "first").clone()
    second = A.attend_paged(obj2, other.q, other.k, other.v)
    for i in range(50):
        assert torch.equal(first, A.attend_paged(obj, b.q, b.k, b.v))
        if i % 10 == 0:
            assert torch.equal(second, A.attend_paged(obj2, other.q, other.k, other.v))
    assert A.attn_get_status() == 0


@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (7, 1, 64), (16, 1, 128)])
def test_rows_of_few_sequences_among_many_empty_ones(cuda_lib, H, G, D):
    """No more rows than sequences, but several of one sequence (the single-token kernel's row blocks)."""
    new = [0] * 12 + [7] + [0] * 5 + [1, 9] + [0] * 10
    kv = [5] * 12 + [300] + [0] * 5 + [70, 9] + [3] * 10
    check(cuda_lib, Batch(new, kv, H, G, D, 16, BF16, seed=41), "few of many")


@pytest.mark.parametrize("D", [64, 128, 80])
def test_the_most_sequences(cuda_lib, D):
    n = 16384
    kv = [1 + (i * 5) % 9 for i in range(n)]
    b = Batch([1] * n, kv, 2, 1, D, 8, F16, seed=42)
    got = cuda_lib.attend_paged(b.object(cuda_lib), b.q, b.k, b.v)
    assert cuda_lib.attn_get_status() == 0
    pick = list(range(0, n, 997)) + [n - 1]
    for i in pick:
        sl = b.slots(i, 0, kv[i])
        k, v = b.k[sl].double(), b.v[sl].double()
        w = torch.softmax(b.q[i].double().view(2, D) @ k.t() / D ** 0.5, -1)
        ref, mag = (w @ v).view(-1), (w @ v.abs()).view(-1)
        assert ((got[i].double() - ref).abs() <= attend_tolerance(ref, mag, F16, 9)).all(), i


def test_infinite_scores_stay_in_their_row(cuda_lib):
    """A NaN query makes its own row NaN and no other; a NaN key within reach makes its sequence's rows NaN."""
    for new in ([1, 1, 1], [40, 40, 40], [400, 400, 400]):
        b = Batch(new, [500, 450, 600], 8, 2, 128, 16, BF16, seed=43)
        want = cuda_lib.attend_paged(b.object(cuda_lib), b.q, b.k, b.v).clone()
        row = b.starts[1]
        b.q[row] = float("nan")
        b.k[b.slots(2, 0, 1)] = float("nan")
        got = cuda_lib.attend_paged(b.object(cuda_lib), b.q, b.k, b.v)
        torch.cuda.synchronize()
        assert cuda_lib.attn_get_status() == 0
        assert torch.isnan(got[row].float()).all() and torch.isnan(got[b.starts[2]:].float()).all()
        keep = [i for i in range(b.starts[2]) if i != row]
        assert torch.equal(got[keep], want[keep])


def test_two_batches_on_two_streams(cuda_lib):
    """Different batch objects (workspaces) may run at the same time."""
    A = cuda_lib
    bs = [Batch([1] * 9, [2000] * 9, 32, 8, 128, 16, BF16, seed=44), Batch([300, 2], [900, 4000], 8, 2, 128, 64, BF16, seed=45)]
    want = [A.attend_paged(b.object(A), b.q, b.k, b.v) for b in bs]
    objs, streams = [b.object(A) for b in bs], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(b.q) for _ in range(20)] for b in bs]
    torch.cuda.synchronize()
    for i in range(20):
        for b, o, s, out in zip(bs, objs, streams, outs):
            A.attend_paged(o, b.q, b.k, b.v, out=out[i], stream=s)
    torch.cuda.synchronize()
    assert A.attn_get_status() == 0
    for w, out in zip(want, outs):
        for o in out:
            assert torch.equal(w, o)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [700, 5, 90]), ([300, 70], [900, 70])])
def test_negative_scale_with_a_cap(cuda_lib, D, new, kv):
    """Scores far past the cap on both sides, turned around by the scale."""
    check(cuda_lib, Batch(new, kv, 8, 2, D, 32, BF16, seed=61), "negative", scale=-0.5, softcap=2.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [700, 5, 90]), ([300, 70], [900, 70])])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(softcap=5.0), dict(softcap=30.0, window=50)])
def test_bits_do_not_depend_on_unattended_positions(cuda_lib, D, new, kv, kw, dtype):
    """Past the end of each sequence the pages hold NaN, zeros or large values: the same bits come out."""
    outs = []
    for junk in (float("nan"), 0.0, 3e4):
        b = Batch(new, kv, 8, 2, D, 32, dtype, seed=62, junk=junk)
        outs.append(cuda_lib.attend_paged(b.object(cuda_lib), b.q, b.k, b.v, **kw))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])



def test_results_made_on_another_stream(cuda_lib):
    """Tensors that a call makes for its results belong to the call's stream, whatever the current one still does."""
    A = cuda_lib
    b = Batch([1, 40], [400, 250], 8, 2, 64, 32, BF16, seed=63)
    obj, table = b.object(A), A.rope_table(512, 64)
    kn, vn = b.k[:41].clone(), b.v[:41].clone()
    kn[:], vn[:] = 1.0, 2.0
    want = A.attend_paged(obj, b.q, b.k, b.v), A.rope(b.q, table, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)
        got = A.attend_paged(obj, b.q, b.k, b.v, stream=stream), A.rope(b.q, table, 8, stream=stream)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert A.append_paged(obj, kn, vn, b.k, b.v, q=b.q, table=table, stream=side).shape == b.q.shape
    torch.cuda.synchronize()


def same_memory(make, nbytes):
    """Runs make() with `nbytes` of freed memory full of ones at hand, which it may be given."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    return make()


@pytest.mark.parametrize("new,kv", [([1], [9000]), ([8], [9000]), ([300, 2], [6000, 700])])
def test_a_call_on_another_stream_waits_for_the_fresh_workspace(cuda_lib, new, kv):
    """A batch object made while the current stream is busy, used at once on another stream: split items count their
    pieces in the workspace, which must have been zeroed by then."""
    A = cuda_lib
    b = Batch(new, kv, 32, 8, 128, 32, BF16, seed=81)
    want = A.attend_paged(b.object(A), b.q, b.k, b.v)
    nbytes = b.object(A).workspace.numel()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        def make():
            torch.cuda._sleep(20_000_000)
            return b.object(A)
        obj = same_memory(make, nbytes)
        got = [A.attend_paged(obj, b.q, b.k, b.v, stream=stream) for _ in range(2)]
        torch.cuda.synchronize()
        assert A.attn_get_status() == 0
        for x in got:
            assert torch.equal(x, want)


@pytest.mark.parametrize("new,kv", [([1], [9000]), ([8], [9000]), ([300, 2], [6000, 700])])
def test_a_batch_object_may_go_while_its_call_runs_on_another_stream(cuda_lib, new, kv):
    """The workspace of a batch object that is dropped after a launch is not given to the current stream's tensors
    before the call has ended."""
    A = cuda_lib
    b = Batch(new, kv, 32, 8, 128, 32, BF16, seed=82)
    want = A.attend_paged(b.object(A), b.q, b.k, b.v)
    nbytes = b.object(A).workspace.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = []
        for _ in range(5):
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)
            got.append(A.attend_paged(b.object(A), b.q, b.k, b.v, stream=stream))
            for _ in range(20):
                torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert A.attn_get_status() == 0
        for x in got:
            assert torch.equal(x, want)


def test_a_shared_workspace_and_a_captured_call_on_another_stream(cuda_lib):
    A = cuda_lib
    b = Batch([8, 1], [9000, 30], 32, 8, 128, 32, BF16, seed=83)
    obj, other = b.object(A), b.object(A)
    want = A.attend_paged(obj, b.q, b.k, b.v)
    other.workspace = obj.workspace
    side = torch.cuda.Stream()
    out = torch.zeros_like(b.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        A.attend_paged(other, b.q, b.k, b.v, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    side.wait_stream(torch.cuda.current_stream())
    got = A.attend_paged(other, b.q, b.k, b.v, stream=side)
    torch.cuda.synchronize()
    assert A.attn_get_status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("rows,page_rows,D", [(64, 16, 128), (64, 16, 64), (2000, 32, 128), (2000, 16, 64), (2000, 4, 64)])
def test_sequences_that_overlap_by_the_hundred_are_left_out(cuda_lib, rows, page_rows, D):
    """A q_start that goes up and down again gives every second sequence all of the rows: more blocks of rows than the
    batch can have, which are reported and not counted in 32 bits."""
    A, n = cuda_lib, 600
    table = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, rows] * (n // 2) + [0], dtype=torch.int32, device="cuda")
    lens = torch.full((n,), 2 * page_rows, dtype=torch.int32, device="cuda")
    obj = A.PagedBatch(table, starts, lens, 8, 2, D, page_rows)
    q = torch.ones(rows, 8 * D, dtype=BF16, device="cuda")
    pool = torch.ones(page_rows, 2 * D, dtype=BF16, device="cuda")
    out = torch.full_like(q, 5.0)
    A.attend_paged(obj, q, pool, pool, out=out)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    assert (out == 5.0).all()
    obj.q_start = torch.tensor([0] * n + [rows], dtype=torch.int32, device="cuda")
    obj.kv_len = lens.clamp_min(rows)[:n].clone()  # past the capacity, which cuts it: reported, and computed
    A.attend_paged(obj, q, pool, pool, out=out)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG and not (out == 5.0).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new,page_rows,D", [(1, 32, 128), (1, 32, 64), (2, 32, 128), (2, 32, 64), (300, 32, 128),
                                             (1, 4, 64), (2, 4, 128)])
def test_many_small_weights_beside_a_large_one(cuda_lib, new, page_rows, D, dtype):
    """Two keys hold nearly all the weight and zeros in V; 65534 others, e^-18 of them each, hold ones.  Weights are
    rounded once: to half a step, or in fp16, where they carry 2^7, below 2^-21 of the largest by 2^-32 of it each."""
    A, n = cuda_lib, 65536
    seqs = 160 if new < 100 else 60
    table = torch.arange(n // page_rows, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    starts = torch.arange(0, new * seqs + 1, new, dtype=torch.int32, device="cuda")
    obj = A.PagedBatch(table, starts, torch.full((seqs,), n, dtype=torch.int32, device="cuda"), 1, 1, D, page_rows)
    q = torch.zeros(new * seqs, D, dtype=dtype, device="cuda")
    q[:, 0] = 4.5
    k, v = torch.zeros(n, D, dtype=dtype, device="cuda"), torch.ones(n, D, dtype=dtype, device="cuda")
    heavy = [0, n - new]
    k[heavy, 0], v[heavy] = 4.0, 0.0
    got = A.attend_paged(obj, q, k, v, scale=1.0).view(seqs, new, D)
    assert A.attn_get_status() == 0
    light = torch.arange(n - new, n, dtype=torch.float64, device="cuda")[:, None] - 1  # light keys of each row
    w = torch.exp(torch.tensor(-18.0, dtype=torch.float64, device="cuda"))
    ref = light * w / (2 + light * w)
    half = torch.finfo(dtype).eps / 2
    tol = 1.01 * (2 * half + 2.0 ** -12) * ref + (n * 2.0 ** -32 if dtype == F16 else 0.0)
    assert ((got.double() - ref).abs() <= tol).all(), float(((got.double() - ref).abs() / tol).max())


@pytest.mark.parametrize("new,kv", [([1], [9000]), ([300, 2], [6000, 700])])
def test_a_workspace_made_on_another_stream_is_ready_and_held(cuda_lib, new, kv):
    """A batch that takes the workspace of one made on a busy stream waits for its fill there, and holds its memory
    against that stream's later tensors."""
    A = cuda_lib
    b = Batch(new, kv, 32, 8, 128, 32, BF16, seed=84)
    want = A.attend_paged(b.object(A), b.q, b.k, b.v)
    nbytes = b.object(A).workspace.numel()
    side, got = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for kind in ["another batch's", "the caller's"] * 2:
        torch.cuda.empty_cache()
        with torch.cuda.stream(side):
            torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
            torch.cuda._sleep(5_000_000)
            if kind == "another batch's":
                workspace = b.object(A).workspace
            else:
                workspace = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        obj = b.object(A)
        if kind == "the caller's":
            torch.cuda.current_stream().wait_stream(side)
        obj.workspace = workspace
        torch.cuda._sleep(5_000_000)
        got.append(A.attend_paged(obj, b.q, b.k, b.v))
        del obj, workspace
        with torch.cuda.stream(side):
            for _ in range(5):
                torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert A.attn_get_status() == 0
    for x in got:
        assert torch.equal(x, want)
