"""attn_append_paged against a plain 64-bit form, and serving steps of append and
attention together."""
import pytest
import torch

from batch_ref import Batch, attend_tolerance, theta, turn

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def positions(b):
    return torch.cat([torch.arange(n - m, n) for m, n in zip(b.new, b.kv)]).cuda()


def all_slots(b):
    return torch.cat([b.slots(i, n - m, n) for i, (m, n) in enumerate(zip(b.new, b.kv))])


def near(got, ref, x, dtype):
    """fp32 table and arithmetic (at most 8 * 2^-24 max|x|), then one rounding to the type."""
    half = torch.finfo(dtype).eps / 2
    tol = half * ref.abs() + 8 * 2.0 ** -24 * (1 + half) * x.double().abs().max() + \
        torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert ((got.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,cache", [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("H,G,D,R,page_rows", [
    (8, 2, 64, 64, 16), (32, 8, 128, 128, 64), (5, 5, 96, 48, 24), (6, 3, 80, 20, 7), (0, 2, 64, 32, 16),
    (4, 1, 33, 2, 5), (2, 2, 40, 0, 1)])
def test_append(cuda_lib, H, G, D, R, page_rows, src, cache, interleaved):
    A = cuda_lib
    b = Batch([3, 0, 1, 50, 1, 17], [3, 9, 90, 70, 1, 33], max(H, G), G, D, page_rows, cache, seed=D, pad=4)
    rows = b.starts[-1]
    g = torch.Generator(device="cuda").manual_seed(3)
    # Columns behind the heads belong to someone else: rows are strided.
    k, v = (torch.randn(b.rows, G * D + 8, generator=g, device="cuda").to(src)[:, :G * D] for _ in range(2))
    q = torch.randn(b.rows, H * D + 16, generator=g, device="cuda").to(src)[:, :H * D] if H else None
    table = A.rope_table(90, R) if R else None
    before_k, before_v = b.k.clone(), b.v.clone()
    q_out = torch.full((b.rows, H * D), 7.0, dtype=cache, device="cuda") if H else None
    got = A.append_paged(b.object(A), k, v, b.k, b.v, q=q, q_out=q_out, table=table, rot_dim=R or None,
                         interleaved=interleaved)
    torch.cuda.synchronize()
    assert A.attn_get_status() == 0
    pos, sl = positions(b), all_slots(b)
    th = theta(R)
    near(b.k[sl], turn(k[:rows].reshape(rows, G, D), pos, th, interleaved).view(rows, -1), k, cache)
    assert torch.equal(b.v[sl], v[:rows].to(cache))
    if H:
        near(got[:rows], turn(q[:rows].reshape(rows, H, D), pos, th, interleaved).view(rows, -1), q, cache)
        assert (got[rows:] == 7.0).all()
    before_k[sl], before_v[sl] = b.k[sl], b.v[sl]  # every other row keeps its bits (NaN among them)
    bits = torch.int32 if cache == F32 else torch.int16
    assert torch.equal(before_k.view(bits), b.k.view(bits)) and torch.equal(before_v.view(bits), b.v.view(bits))


@pytest.mark.parametrize("n", [1, 31, 32, 33, 1000, 1025, 40000])
def test_many_sequences(cuda_lib, n):
    """The search of a row's sequence, with sequences that have no rows between."""
    new = [1 if i % 3 else 0 for i in range(n)]
    if sum(new) == 0:
        new[0] = 1
    b = Batch(new, [4] * n, 1, 1, 8, 4, F32, seed=n, junk=0.0)
    rows = b.starts[-1]
    k = torch.arange(rows * 8, device="cuda", dtype=F32).view(rows, 8)
    cuda_lib_batch = cuda_lib.PagedBatch(b.block_table, b.q_start, b.kv_len, 1, 1, 8, 4)
    cuda_lib.append_paged(cuda_lib_batch, k, -k, b.k, b.v)
    assert cuda_lib.attn_get_status() == 0
    seq = torch.tensor([i for i, m in enumerate(new) if m])
    sl = (b.table[seq, 0].long() * 4 + 3).cuda()
    assert torch.equal(b.k[sl], k) and torch.equal(b.v[sl], -k)


def test_bad_device_values_are_reported_and_skipped(cuda_lib):
    A = cuda_lib
    b = Batch([2, 2, 2, 2], [10, 10, 10, 10], 2, 1, 64, 8, BF16, seed=1, junk=0.0, extra_blocks=0)
    table = b.block_table.clone()
    table[0, 1] = 2 ** 31 - 1               # a page outside the pool
    kv = b.dev([10, 1, 10 ** 6, 10])        # before position 0, past the capacity
    k = torch.ones(8, 64, dtype=BF16, device="cuda")
    q = torch.ones(8, 128, dtype=BF16, device="cuda")
    q_out = torch.full_like(q, 5.0)
    keep = b.k.clone()
    A.append_paged(b.object(A, block_table=table, kv_len=kv), k, k, b.k, b.v, q=q, q_out=q_out,
                   table=A.rope_table(16, 64))
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    wrote = (b.k != keep).any(1).nonzero().flatten().tolist()
    want = sorted(b.slots(3, 8, 10).tolist() + b.slots(1, 0, 1).tolist())
    assert wrote == want
    assert (q_out[[0, 1, 2, 4, 5]] == 5.0).all() and (q_out[[3, 6, 7]] != 5.0).any(1).all()
    # A position past the table.
    A.append_paged(b.object(A), k, k, b.k, b.v, table=A.rope_table(9, 64))
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    # Rows behind a q_start that passes them belong to no sequence.
    A.append_paged(b.object(A, q_start=b.dev([8, 8, 8, 8, 8])), k, k, b.k, b.v)
    assert A.attn_get_status() == 0


def test_fp32_pools_serve_the_single_sequence_calls(cuda_lib, orc):
    """An fp32 append fills the pool that attn_decode_paged reads."""
    import numpy as np
    A = cuda_lib
    H, G, D, pr, n = 8, 2, 64, 32, 100
    b = Batch([n], [n], H, G, D, pr, F32, seed=4, extra_blocks=0)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(n, G * D, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(1, H * D, generator=g, device="cuda")
    A.append_paged(b.object(A), k, v, b.k, b.v)
    ws = torch.zeros(A.attn_decode_workspace_bytes(H, G, D, pr * b.max_blocks), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    A.attn_decode_paged(q, b.k, b.v, b.block_table[0].contiguous(), b.dev([n - 1]), out, H, G, D, pr, b.num_pages,
                        b.max_blocks, ws)
    ref = orc.decode(q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), n - 1, H, G, D, n)
    assert np.abs(out.cpu().numpy() - ref).max() <= 1e-5 + 1e-4 * np.abs(ref).max()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompt_chunks_then_single_tokens(cuda_lib, dtype):
    """Serving as a program runs it: prompts in chunks, then single tokens (captured once and replayed), each
    step an append with Q and K turned and the attention over the pages; against the whole sequences in 64 bits,
    from the values the cache holds."""
    A = cuda_lib
    H, G, D, pr, S = 8, 2, 64, 16, 3
    total = [70, 41, 130]
    b = Batch([1] * S, total, H, G, D, pr, dtype, seed=6)
    g = torch.Generator(device="cuda").manual_seed(7)
    table = A.rope_table(256, D)
    obj = b.object(A)
    data = [[torch.randn(n, w * D, generator=g, device="cuda").to(dtype) for w in (H, G, G)] for n in total]
    outs = [torch.zeros(n, H * D, device="cuda", dtype=torch.float64) for n in total]
    turned = [torch.zeros(n, H * D, device="cuda", dtype=dtype) for n in total]

    def step(cuts, run):
        """One step of rows [lo, hi) of each sequence."""
        starts = [0]
        for lo, hi in cuts:
            starts.append(starts[-1] + hi - lo)
        b.q_start.copy_(b.dev(starts))
        b.kv_len.copy_(b.dev([hi for _, hi in cuts]))
        q, k, v = (torch.cat([data[i][x][lo:hi] for i, (lo, hi) in enumerate(cuts)]) for x in range(3))
        qt, o = run(q, k, v)
        for i, (lo, hi) in enumerate(cuts):
            outs[i][lo:hi] = o[starts[i]:starts[i + 1]].double()
            turned[i][lo:hi] = qt[starts[i]:starts[i + 1]]

    def eager(q, k, v):
        qt = A.append_paged(obj, k, v, b.k, b.v, q=q, table=table)
        return qt, A.attend_paged(obj, qt, b.k, b.v)

    step([(0, 30), (0, 0), (0, 64)], eager)
    step([(30, 35), (0, 33), (64, 122)], eager)
    done = [35, 33, 122]
    fq, fk, fv = (torch.zeros(S, w * D, dtype=dtype, device="cuda") for w in (H, G, G))
    fqt, fo = torch.zeros_like(fq), torch.zeros_like(fq)

    def both():
        A.append_paged(obj, fk, fv, b.k, b.v, q=fq, q_out=fqt, table=table)
        A.attend_paged(obj, fqt, b.k, b.v, out=fo)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    b.q_start.copy_(b.dev([0, 1, 2, 3]))
    b.kv_len.copy_(b.dev([n + 1 for n in done]))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        both()

    def replay(q, k, v):
        fq.copy_(q), fk.copy_(k), fv.copy_(v)
        graph.replay()
        return fqt, fo

    for t in range(8):
        step([(n + t, n + t + 1) for n in done], replay)
    torch.cuda.synchronize()
    assert A.attn_get_status() == 0
    b.kv = [n + 8 for n in done]
    b.new = list(b.kv)
    b.starts = [0, b.kv[0], b.kv[0] + b.kv[1], sum(b.kv)]
    q = torch.cat([t[:n] for t, n in zip(turned, b.kv)])
    got = torch.cat([o[:n] for o, n in zip(outs, b.kv)])
    pos = torch.cat([torch.arange(n, device="cuda") for n in b.kv])
    raw = torch.cat([data[i][0][:n] for i, n in enumerate(b.kv)])
    near(q, turn(raw.view(-1, H, D), pos, theta(D), False).view(-1, H * D), raw, dtype)
    ref, mag = b.attend(q=q)
    assert ((got - ref).abs() <= attend_tolerance(ref, mag, dtype, 130)).all()


def test_refusals(cuda_lib):
    A = cuda_lib
    b = Batch([1], [20], 4, 2, 64, 16, BF16, seed=14)
    obj, k = b.object(A), torch.zeros(1, 128, dtype=BF16, device="cuda")
    for kw in (dict(k_new=k[:, :64]), dict(v_new=k.float()), dict(q=k), dict(k_pages=b.k[:-1], v_pages=b.v[:-1]),
               dict(table=A.rope_table(32, 64), rot_dim=32), dict(k_new=k.cpu())):
        args = dict(k_new=k, v_new=k, k_pages=b.k, v_pages=b.v)
        args.update(kw)
        with pytest.raises(ValueError):
            A.append_paged(obj, **args)
    with pytest.raises(A.AttnError):  # bf16 rows into an fp32 cache
        A.append_paged(obj, k, k, b.k.float(), b.v.float())


@pytest.mark.parametrize("src,cache", [(BF16, BF16), (F32, F16)])
def test_a_result_the_call_makes_holds_zeros_where_no_row_is_written(cuda_lib, src, cache):
    """Rows behind the last sequence, and rows that are skipped, in a padded batch's q: zeros as attend_paged gives,
    not what the memory held before."""
    A = cuda_lib
    b = Batch([2, 3], [10, 20], 4, 2, 64, 16, cache, seed=9, pad=6, junk=0.0)
    k, v, q = (torch.ones(b.rows, w * 64, dtype=src, device="cuda") for w in (2, 2, 4))
    for lens, skipped in (([10, 20], []), ([1, 20], [0])):
        obj = b.object(A, kv_len=b.dev(lens))
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.full((b.rows, 4 * 64), 7.0, dtype=cache, device="cuda")
        got = A.append_paged(obj, k, v, b.k, b.v, q=q)
        assert A.attn_get_status() == (A.ATTN_ERR_INVALID_ARG if skipped else 0)
        want = torch.ones(b.rows, 4 * 64, dtype=cache, device="cuda")
        want[skipped + list(range(5, b.rows))] = 0.0
        assert torch.equal(got, want)
