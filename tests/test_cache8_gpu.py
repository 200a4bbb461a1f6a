"""The 8-bit paged cache: append and read-back against plain 64-bit forms."""
import pytest
import torch

from batch_ref import theta, turn
from cache8_ref import Batch8, decode, encode, exp_for

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def positions(b):
    return torch.cat([torch.arange(n - m, n) for m, n in zip(b.new, b.kv)]).cuda()


def rows_of(b, heads, src, seed, pad=8, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = scale * torch.randn(b.rows, heads * b.D + pad, generator=g, device="cuda")
    return x.to(src)[:, :heads * b.D]


def norm64(x, w):
    x = x.double()
    return x if w is None else x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()


def check_cache(b, before, name, x, rel):
    """`before`: codes and scales before the call; x [rows, G, D] in 64 bits; rel: the kernel's values may be off by
    rel of the largest of their head (a scale may then be that of a neighbouring size, a code its neighbour)."""
    codes, scales = before
    G, D = b.G, b.D
    want_codes, want_scales = codes.clone(), scales.clone()
    got_codes, got_scales = b.codes[name], b.scales[name]
    starts = dict(zip(range(len(b.new)), b.starts))
    for i, first, held, end in b.groups():
        slots = b.slots(i, first, first + end)
        blk = int(slots[0]) // b.sr
        row0 = starts[i] + first + held - (b.kv[i] - b.new[i])
        new = x[row0:row0 + end - held]
        amax = new.abs().amax((0, 2))
        e0 = scales[blk].double().clamp(113, 134) - 127 if held else torch.full((G,), -14.0, device="cuda").double()
        e = got_scales[blk].double() - 127
        lo, hi = (torch.maximum(e0, exp_for(amax * (1 + s * 2 * rel))) for s in (-1, 1))
        assert ((e == lo) | (e == hi)).all()
        size = torch.exp2(e)[None, :, None]
        old = decode(codes[slots[:held], :G * D]).view(held, G, D) * torch.exp2(e0 - e)[None, :, None]
        assert torch.equal(decode(got_codes[slots[:held], :G * D]).view(held, G, D), encode(old))
        got = decode(got_codes[slots[held:], :G * D]).view(-1, G, D)
        if rel == 0:
            assert torch.equal(got, encode(new / size))
        else:
            # Half a step of a code (2^-4 of it, 2^-10 below 2^-6) of the value that the kernel rounded.
            off = rel * 2 * new.abs().amax(-1, keepdim=True)
            tol = off + size * torch.maximum((new.abs() + off) / size * 2.0 ** -4, torch.full_like(new, 2.0 ** -10))
            assert ((got * size - new).abs() <= tol).all()
        want_codes[slots, :G * D] = got_codes[slots, :G * D]
        want_scales[blk] = got_scales[blk]
    # Everything else keeps its bits.
    assert torch.equal(want_codes, got_codes) and torch.equal(want_scales, got_scales)


CASES = [  # new, kv, H, G, D, R, page_rows, scale_rows
    ([3, 0, 1, 50, 1, 17], [3, 9, 90, 70, 1, 33], 8, 2, 64, 64, 16, 16),
    ([3, 0, 1, 50, 1, 17], [3, 9, 90, 70, 1, 33], 32, 8, 128, 128, 64, 32),
    ([5, 130, 1], [6, 131, 500], 5, 5, 96, 48, 24, 8),
    ([40, 1, 1, 7], [41, 1, 8, 300], 6, 3, 80, 20, 7, 7),
    ([9, 2, 64], [10, 300, 64], 0, 2, 64, 32, 16, 1),
    ([1] * 40, list(range(1, 41)), 4, 1, 16, 2, 10, 5),
    ([300, 1], [777, 3], 2, 2, 48, 0, 256, 256),
    ([129], [1029], 3, 1, 128, 64, 128, 128),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,normed", [(F32, False), (F32, True), (BF16, False), (BF16, True), (F16, True)])
@pytest.mark.parametrize("new,kv,H,G,D,R,page_rows,scale_rows", CASES)
def test_append(cuda_lib, new, kv, H, G, D, R, page_rows, scale_rows, src, normed, interleaved):
    A = cuda_lib
    b = Batch8(new, kv, max(H, G), G, D, page_rows, scale_rows, seed=D, pad=4, kv_dim=G * D + 16)
    rows = b.starts[-1]
    k, v = rows_of(b, G, src, 3), rows_of(b, G, src, 4)
    q = rows_of(b, H, src, 5, pad=16) if H else None
    g = torch.Generator(device="cuda").manual_seed(6)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(src) if normed else None for _ in range(2))
    wq = wq if H else None
    table = A.rope_table(max(kv), R) if R else None
    q_out = torch.full((b.rows, H * D), 7.0, dtype=BF16 if src == F32 else src, device="cuda") if H else None
    before = {x: (b.codes[x].clone(), b.scales[x].clone()) for x in "kv"}
    A.append_paged8(b.object(A), k, v, b.cache(A), q=q, q_out=q_out, table=table, rot_dim=R or None,
                    interleaved=interleaved, q_weight=wq, k_weight=wk)
    assert A.attn_get_status() == 0
    pos, th = positions(b), theta(R)
    # fp32 arithmetic, as in the norm's and the turn's own tests.
    rel = (D * 2.0 ** -25 + 2.0 ** -22 if normed else 0.0) + (8 * 2.0 ** -24 if R or normed else 0.0)
    check_cache(b, before["v"], "v", v[:rows].double().reshape(rows, G, D), 0.0)
    check_cache(b, before["k"], "k", turn(norm64(k[:rows].reshape(rows, G, D), wk), pos, th, interleaved), rel)
    if H:
        z = norm64(q[:rows].reshape(rows, H, D), wq)
        ref = turn(z, pos, th, interleaved)
        half = torch.finfo(q_out.dtype).eps / 2
        tol = half * ref.abs() + (1 + half) * (rel + 2.0 ** -24) * 3 * z.abs().amax(-1, keepdim=True) + 1e-12
        assert ((q_out[:rows].double().view(rows, H, D) - ref).abs() <= tol + torch.finfo(q_out.dtype).tiny).all()
        assert (q_out[rows:] == 7.0).all()


def test_token_by_token_equals_one_call_but_for_subnormal_codes(cuda_lib):
    """A block's scale grows as larger rows come; codes follow it without a second rounding while they are normal."""
    A = cuda_lib
    n, G, D = 64, 2, 64
    x = torch.randn(n, G * D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x *= torch.exp2(torch.linspace(-6, 4, n, device="cuda"))[:, None]  # ever larger
    one = Batch8([n], [n], 2, G, D, 16, 16, seed=2)
    A.append_paged8(one.object(A), x, x, one.cache(A))
    step = Batch8([1], [n], 2, G, D, 16, 16, seed=2)
    batch, cache = step.object(A), step.cache(A)
    for t in range(n):
        step.kv_len.fill_(t + 1)
        A.append_paged8(batch, x[t:t + 1], x[t:t + 1], cache)
    sl = one.slots(0, 0, n)
    assert torch.equal(one.scales["k"], step.scales["k"])
    size = torch.exp2(one.scales["k"][sl // 16].double() - 127).repeat_interleave(D, 1)
    a, b = decode(one.codes["k"][sl]) * size, decode(step.codes["k"][sl]) * size
    # A code that became subnormal (below 2^-6) was rounded once more at each growth, by at most half of the step 2^-9
    # that each scale had: below twice the last one's.
    assert torch.equal(a[a.abs() >= 2.0 ** -6 * size], b[a.abs() >= 2.0 ** -6 * size])
    assert ((a - b).abs() <= 2.0 ** -9 * size).all()


def test_extreme_values(cuda_lib):
    """Zeros, magnitudes past the largest scale, infinities and NaN, values at a scale's border."""
    A = cuda_lib
    G, D, sr = 1, 16, 4
    b = Batch8([40], [40], 1, G, D, 8, sr, seed=3)
    x = torch.zeros(40, D, device="cuda")
    x[4:8] = torch.linspace(-1, 1, D, device="cuda") * 1e-9
    x[8, 3], x[9, 0] = 1e9, 1.0
    x[12, 5], x[13, 1] = float("inf"), -float("inf")
    x[16, 2], x[17, 2] = float("nan"), 3.0
    x[20] = 448.0
    x[24, 0], x[25, 1] = 448.0 * (1 + 2.0 ** -20), 1.0
    x[28, 0] = 448.0 * 2.0 ** 7
    x[32, 0], x[33, 0] = 448.0 * 2.0 ** -14, 2.0 ** -24
    x[36, 0], x[37, 0] = 449.0 * 2.0 ** -14, 3 * 2.0 ** -24
    A.append_paged8(b.object(A), x, x, b.cache(A))
    sl = b.slots(0, 0, 40)
    scales = b.scales["v"][sl[::sr] // sr, 0].tolist()
    assert [s - 127 for s in scales] == [-14, -14, 7, 7, -7, 0, 1, 7, -14, -13]
    assert torch.equal(b.codes["k"], b.codes["v"]) and torch.equal(b.scales["k"], b.scales["v"])
    got = b.values("v")[sl]
    assert (got[0:4] == 0).all() and (got[4:8] == 0).all() and got[8, 3] == 57344 and got[12, 5] == 57344
    assert got[13, 1] == -57344 and got[16, 2].isnan() and got[17, 2] == 3.0 and (got[20] == 448.0).all()
    assert got[24, 0] == 448.0 and got[28, 0] == 57344 and got[32, 0] == 448 * 2.0 ** -14 and got[33, 0] == 0
    assert got.isnan().sum() == 1


def test_bad_device_values_are_reported_and_skipped(cuda_lib):
    A = cuda_lib
    b = Batch8([2, 2, 2, 2], [10, 10, 10, 10], 2, 1, 64, 8, 4, seed=1, extra_blocks=0)
    before = b.codes["k"].clone(), b.scales["k"].clone()
    table = b.block_table.clone()
    table[0, 1] = 2 ** 31 - 1               # a page outside the pool
    kv = b.dev([10, 1, 10 ** 6, 10])        # before position 0, past the capacity
    k, q = torch.ones(8, 64, dtype=BF16, device="cuda"), torch.ones(8, 128, dtype=BF16, device="cuda")
    q_out = torch.full_like(q, 5.0)
    rope = A.rope_table(16, 64)
    A.append_paged8(b.object(A, block_table=table, kv_len=kv), k, k, b.cache(A), q=q, q_out=q_out, table=rope)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    changed = (b.codes["k"] != before[0]).any(1).nonzero().flatten().tolist()
    assert changed == sorted(b.slots(3, 8, 10).tolist() + b.slots(1, 0, 1).tolist())
    assert (q_out[[0, 1, 2, 4, 5]] == 5.0).all() and (q_out[[3, 6, 7]] != 5.0).any(1).all()
    blocks = (b.scales["k"] != before[1]).any(1).nonzero().flatten().tolist()
    assert set(blocks) <= {int(b.slots(3, 8, 9)[0]) // 4, int(b.slots(1, 0, 1)[0]) // 4}
    # A position past the rotary table: its rows alone are left out.
    c = Batch8([6], [10], 2, 1, 64, 8, 4, seed=1)
    keep = c.codes["k"].clone()
    A.append_paged8(c.object(A), k[:6], k[:6], c.cache(A), table=A.rope_table(9, 64))
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    changed = (c.codes["k"] != keep).any(1).nonzero().flatten().tolist()
    assert changed == sorted(c.slots(0, 4, 9).tolist())
    # Rows behind a q_start that passes them, and no rows at all.
    keep = b.codes["k"].clone()
    A.append_paged8(b.object(A, q_start=b.dev([8, 8, 8, 8, 8])), k, k, b.cache(A))
    A.append_paged8(b.object(A), k[:0], k[:0], b.cache(A))
    assert A.attn_get_status() == 0 and torch.equal(keep, b.codes["k"])


@pytest.mark.parametrize("n", [1, 33, 1000, 20000])
@pytest.mark.parametrize("per", [1, 5])
def test_many_sequences(cuda_lib, n, per):
    """The search of a row's sequence, with sequences that have no rows between."""
    A = cuda_lib
    new = [per if i % 7 == 3 or n == 1 else 0 for i in range(n)]
    b = Batch8(new, [7] * n, 1, 1, 16, 8, 8, seed=n)
    rows = b.starts[-1]
    x = torch.randn(rows, 16, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    before = b.codes["v"].clone(), b.scales["v"].clone()
    A.append_paged8(b.object(A), x, x, b.cache(A))
    assert A.attn_get_status() == 0
    seq = torch.tensor([i for i, m in enumerate(new) for _ in range(m)])
    pos = torch.tensor([7 - per + j for m in new for j in range(m)])
    sl = (b.table[seq, 0].long() * 8 + pos).cuda()
    size = torch.exp2(b.scales["v"][sl // 8].double() - 127)
    assert torch.equal(decode(b.codes["v"][sl]), encode(x.double() / size))
    amax = x.double().abs().view(-1, per, 16).amax((1, 2))
    held = before[1][sl[::per] // 8, 0].double() - 127
    assert torch.equal(b.scales["v"][sl[::per] // 8, 0].double() - 127,
                       torch.maximum(held, exp_for(amax)) if per < 7 else exp_for(amax))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("kv,first,G,D,page_rows,scale_rows", [
    ([1, 90, 17], None, 2, 64, 16, 16), ([5000, 1, 300], [17, 0, 300], 8, 128, 64, 8), ([33, 70], [32, 1], 3, 80, 24, 1),
    ([20, 41, 9], [0, 40, 3], 1, 48, 10, 5)])
def test_read(cuda_lib, kv, first, G, D, page_rows, scale_rows, dtype):
    A = cuda_lib
    b = Batch8([0] * len(kv), kv, G, G, D, page_rows, scale_rows, seed=4, kv_dim=G * D + 32)
    counts = [n - f for n, f in zip(kv, first or [0] * len(kv))]
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    for pad in (0, 8, 3):  # (3: rows that do not begin on 16 bytes)
        k, v = (torch.full((starts[-1] + 2, G * D + pad), 9.0, dtype=dtype, device="cuda")[:, :G * D] for _ in range(2))
        A.read_paged8(b.object(A), b.cache(A), b.dev(starts), k, v, first=b.dev(first) if first else None)
        assert A.attn_get_status() == 0
        sl = torch.cat([b.slots(i, n - c, n) for i, (n, c) in enumerate(zip(kv, counts))])
        for name, got in (("k", k), ("v", v)):
            assert torch.equal(got[:-2].double(), b.values(name)[sl])
            assert (got[-2:] == 9.0).all()


def test_read_of_bad_positions(cuda_lib):
    A = cuda_lib
    b = Batch8([0, 0], [10, 12], 1, 1, 16, 8, 8, seed=5)
    table = b.block_table.clone()
    table[1, 0] = b.num_pages
    out = [torch.full((14, 16), 9.0, device="cuda") for _ in range(2)]
    starts = b.dev([1, 5, 13])  # positions 8 .. 11 of the first, 6 .. 13 of the second
    A.read_paged8(b.object(A, block_table=table), b.cache(A), starts, *out, first=b.dev([8, 6]))
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    for name, x in zip("kv", out):
        assert (x[0] == 9.0).all() and (x[13] == 9.0).all()
        assert torch.equal(x[1:3].double(), b.values(name)[b.slots(0, 8, 10)]) and (x[3:5] == 0).all()
        assert (x[5:7] == 0).all() and (x[11:13] == 0).all()
        assert torch.equal(x[7:11].double(), b.values(name)[b.slots(1, 8, 12)])


def test_streams_and_graphs(cuda_lib):
    A = cuda_lib
    b = Batch8([1] * 20, list(range(5, 25)), 4, 2, 64, 16, 16, seed=6)
    x, q = rows_of(b, 2, BF16, 1, pad=0), rows_of(b, 4, BF16, 2, pad=0)
    w = torch.ones(64, device="cuda", dtype=BF16)
    rope = A.rope_table(64, 64)
    start = {n: (b.codes[n].clone(), b.scales[n].clone()) for n in "kv"}

    def reset():
        for n in "kv":
            b.codes[n].copy_(start[n][0])
            b.scales[n].copy_(start[n][1])

    batch, cache = b.object(A), b.cache(A)
    rows = sum(b.kv)
    starts = b.dev([sum(b.kv[:i]) for i in range(21)])
    k1, v1, k2, v2 = (torch.zeros(rows, 128, device="cuda") for _ in range(4))
    q1 = A.append_paged8(batch, x, x, cache, q=q, table=rope, q_weight=w, k_weight=w)
    A.read_paged8(batch, cache, starts, k1, v1)
    reset()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q2 = A.append_paged8(batch, x, x, cache, q=q, table=rope, q_weight=w, k_weight=w, stream=side)
    A.read_paged8(batch, cache, starts, k2, v2, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(q1, q2) and torch.equal(k1, k2) and torch.equal(v1, v2)
    reset()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q2 = A.append_paged8(batch, x, x, cache, q=q, table=rope, q_weight=w, k_weight=w)
        A.read_paged8(batch, cache, starts, k2, v2)
    k2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(k1, k2) and torch.equal(v1, v2)


@pytest.mark.parametrize("src,pad", [(F32, 0), (BF16, 8), (F16, 0), (BF16, 3)])  # (3: rows that do not begin on 16 bytes)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 64), (64, 16), (96, 48), (128, 0), (64, 0)])
def test_infinities_stay_in_columns_that_do_not_turn(cuda_lib, D, R, interleaved, src, pad):
    """They become 57344 in the cache and stay infinities in Q; the columns beside them are as without them, but for the
    scale of their block."""
    A = cuda_lib
    n, H, G, sr = 24, 4, 2, 4
    b = Batch8([n], [n], H, G, D, 8, sr, seed=D)
    k, v, q = rows_of(b, G, src, 1, pad), rows_of(b, G, src, 2, pad), rows_of(b, H, src, 3, pad)
    inf = float("inf")
    where = [(4 * i + 1, D + c, inf if i % 2 else -inf) for i, c in enumerate((R, R + 3, R + 9, D - 1))]
    for row, col, x in where:
        k[row, col] = v[row, col] = x
        q[row, D + col] = x
    table = A.rope_table(n, R) if R else None
    out = A.append_paged8(b.object(A), k, v, b.cache(A), q=q, table=table, rot_dim=R or None, interleaved=interleaved)
    assert A.attn_get_status() == 0
    pos, th = positions(b), theta(R)
    sl = b.slots(0, 0, n)
    hit = torch.zeros(n, G * D, dtype=torch.bool, device="cuda")
    for row, col, x in where:
        hit[row, col] = True
    for name, x in (("k", turn(k.reshape(n, G, D), pos, th, interleaved)), ("v", v.double().reshape(n, G, D))):
        got = b.values(name)[sl]
        assert got.isfinite().all()
        x = x.reshape(n, -1)
        assert torch.equal(got[hit], torch.sign(x[hit]) * 57344)
        scales = b.scales[name][sl[::sr] // sr].double() - 127
        infinite = hit.view(-1, sr, G, D).any(1).any(-1)
        amax = torch.where(hit, torch.zeros_like(x), x).abs().view(-1, sr, G, D).amax((1, 3))
        low, high = exp_for(amax * (1 - 2.0 ** -20)), exp_for(amax * (1 + 2.0 ** -20))  # (eight roundings of fp32)
        assert (scales[infinite] == 7).all() and ((scales == low) | (scales == high) | infinite).all()
        size = torch.exp2(scales).repeat_interleave(sr, 0).repeat_interleave(D, 1)
        tol = 2.0 ** -20 + torch.maximum(x.abs() * 1.001 * 2.0 ** -4, size * 2.0 ** -10)
        assert ((got - x).abs() <= tol)[~hit].all()
    ref = turn(q.reshape(n, H, D), pos, th, interleaved).reshape(n, -1)
    assert torch.equal(out.isinf(), ref.isinf()) and not out.isnan().any()
    fine = ref.isfinite()
    # (A result is made of two values, of up to 6 here.)
    assert torch.equal(out[~fine].double(), ref[~fine])
    assert ((out.double() - ref).abs() <= torch.finfo(out.dtype).eps / 2 * ref.abs() + 2.0 ** -18)[fine].all()


def test_calls_without_rows(cuda_lib):
    """Q, K and V of no rows, through the package: results of no rows, and an unchanged cache; nor any rows read."""
    A = cuda_lib
    b = Batch8([0, 0], [5, 9], 4, 2, 64, 8, 8, dtype=BF16, seed=3)
    w, table = torch.ones(64, dtype=BF16, device="cuda"), A.rope_table(16, 64)
    q, k, v = (torch.empty(0, n * 64, dtype=BF16, device="cuda") for n in (4, 2, 2))
    before = [x.clone() for d in (b.codes, b.scales) for x in d.values()]
    batch, cache = b.object(A), b.cache(A)
    out = A.append_paged8(batch, k, v, cache, q=q, table=table, q_weight=w, k_weight=w)
    assert out.shape == (0, 256)
    assert A.append_paged8(batch, k, v, cache, q=q, q_out=out, table=table) is out
    assert A.attend_paged8(batch, out, cache, window=4, sinks=1).shape == (0, 256)
    A.read_paged8(batch, cache, b.dev([0, 0, 0]), k, v)
    assert all(torch.equal(x, y) for x, y in zip(before, [x for d in (b.codes, b.scales) for x in d.values()]))
    pools = torch.zeros_like(b.k), torch.zeros_like(b.v)
    out = A.append_paged(batch, k, v, *pools, q=q, table=table)
    assert out.shape == (0, 256) and A.attend_paged(batch, out, *pools).shape == (0, 256)
    assert A.attn_get_status() == 0


@pytest.mark.parametrize("page_rows,scale_rows", [(64, 16), (7, 1)])
def test_pools_whose_offsets_pass_32_bits(cuda_lib, page_rows, scale_rows):
    """Pages behind byte 2^31 of a pool, and behind scale 2^24: the bits of the same step over a small pool."""
    A = cuda_lib
    G, D, H = 8, 128, 16
    new, kv = [1, 200, 3], [40, 210, 90]
    b = Batch8(new, kv, H, G, D, page_rows, scale_rows, dtype=BF16, seed=4)
    pages = 2 ** 31 // (page_rows * G * D) + 1 + b.num_pages
    far = pages - b.num_pages
    x, q = rows_of(b, G, BF16, 1, pad=0), rows_of(b, H, BF16, 2, pad=0)
    w, rope = torch.ones(D, device="cuda", dtype=BF16), A.rope_table(256, D)
    starts = b.dev([0, 40, 250, 340])
    results = []
    for shift, total in ((0, b.num_pages), (far, pages)):
        cache = A.PagedCache8(*(torch.empty(total * page_rows, G * D, dtype=torch.uint8, device="cuda") for _ in "kv"),
                              *(torch.empty(total * page_rows // scale_rows, G, dtype=torch.uint8, device="cuda") for _ in "kv"))
        for pool, n in ((cache.k_pages, "k"), (cache.v_pages, "v")):
            pool[shift * page_rows:] = b.codes[n]
        for pool, n in ((cache.k_scales, "k"), (cache.v_scales, "v")):
            pool[shift * page_rows // scale_rows:] = b.scales[n]
        batch = b.object(A, block_table=torch.where(b.block_table >= 0, b.block_table + shift, b.block_table))
        one = A.PagedBatch(batch.block_table[:1].contiguous(), b.dev([0, 1]), b.kv_len[:1].contiguous(), H, G, D, page_rows)
        qt = A.append_paged8(batch, x, x, cache, q=q, table=rope, q_weight=w, k_weight=w)
        k, v = (torch.empty(340, G * D, device="cuda") for _ in "kv")
        A.read_paged8(batch, cache, starts, k, v)
        results.append((qt, k, v, A.attend_paged8(batch, qt, cache), A.attend_paged8(one, qt[:1], cache),
                        cache.k_pages[shift * page_rows:].clone(), cache.v_scales[shift * page_rows // scale_rows:].clone()))
        assert A.attn_get_status() == 0
        del cache
    assert all(torch.equal(a, c) for a, c in zip(*results))
