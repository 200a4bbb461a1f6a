"""The C entry points of the head norms, the 8-bit cache and first positions as bound, against the allocating calls over them
(which their own tests hold to 64 bits): the same bits, and the same status from bad sizes."""
import pytest
import torch

from cache8_ref import Batch8

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_norms(cuda_lib):
    A = cuda_lib
    rows, H, G, D = 37, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    q, k, dq, dk, w = mk(rows, H * D), mk(rows, G * D), mk(rows, H * D), mk(rows, G * D), mk(D)
    table = A.rope_table(rows, D)
    want = A.qk_norm_rope(q, k, H, G, w, w, table=table) + A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table)
    got = [torch.empty_like(x) for x in want]
    A.attn_qk_norm_rope(q, k, got[0], got[1], w, w, rows, H, G, D, H * D, G * D, H * D, G * D, 1e-6, rot_dim=D, table=table)
    workspace = torch.empty(A.attn_qk_norm_rope_backward_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    A.attn_qk_norm_rope_backward(dq, dk, q, k, got[2], got[3], w, w, got[4], got[5], rows, H, G, D, H * D, G * D, H * D,
                                 G * D, H * D, G * D, 1e-6, rot_dim=D, table=table, workspace=workspace)
    assert A.attn_get_status() == 0 and all(torch.equal(a, b) for a, b in zip(want, got))
    # K alone; a workspace too small; weights of two types.
    alone = torch.empty_like(k)
    A.attn_qk_norm_rope(None, k, None, alone, None, w, rows, 0, G, D, 0, G * D, 0, G * D, 1e-6, rot_dim=D, table=table)
    assert torch.equal(alone, want[1])
    with pytest.raises(A.AttnError):
        A.attn_qk_norm_rope_backward(dq, dk, q, k, got[2], got[3], w, w, got[4], got[5], rows, H, G, D, H * D, G * D,
                                     H * D, G * D, H * D, G * D, 1e-6, workspace=workspace[:64])
    with pytest.raises(ValueError):
        A.attn_qk_norm_rope(q, k, got[0], got[1], w, w.float(), rows, H, G, D, H * D, G * D, H * D, G * D, 1e-6)


def test_the_weights_gradient_of_a_tensor_that_is_left_out_is_zero(cuda_lib):
    A = cuda_lib
    rows, G, D = 9, 2, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    k, dk = (torch.randn(rows, G * D, generator=g, device="cuda") for _ in range(2))
    w, out = torch.ones(D, device="cuda"), torch.empty_like(k)
    workspace = torch.empty(A.attn_qk_norm_rope_backward_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    one, other = (torch.full((D,), 7.0, device="cuda") for _ in range(2))
    A.attn_qk_norm_rope_backward(None, dk, None, k, None, out, None, w, other, one, rows, 0, G, D, 0, G * D, 0, G * D, 0,
                                 G * D, 1e-6, workspace=workspace)
    assert (other == 0).all() and one.isfinite().all() and (one != 0).any()
    other.fill_(7.0)
    A.attn_qk_norm_rope_backward(dk, None, k, None, out, None, w, None, one, other, rows, G, 0, D, G * D, 0, G * D, 0,
                                 G * D, 0, 1e-6, workspace=workspace)
    assert A.attn_get_status() == 0 and (other == 0).all() and (one != 0).any()


def test_a_serving_step(cuda_lib):
    A = cuda_lib
    H, G, D, pr, sr = 8, 2, 64, 16, 8
    b = Batch8([1, 5, 0, 40], [9, 70, 3, 100], H, G, D, pr, sr, dtype=BF16, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(b.rows, n * D, generator=g, device="cuda").to(BF16) for n in (H, G, G))
    w = 1 + 0.2 * torch.randn(D, generator=g, device="cuda").to(BF16)
    table, batch = A.rope_table(128, D), b.object(A)
    old = [x.clone() for d in (b.codes, b.scales) for x in d.values()]
    cache = A.PagedCache8(*[x.clone() for x in old])
    want_q = A.append_paged8(batch, k, v, cache, q=q, table=table, q_weight=w, k_weight=w)
    want = A.attend_paged8(batch, want_q, cache, window=20, sinks=3)
    starts = b.dev([0, 9, 79, 82, 182])
    ks, vs = A.read_paged8(batch, cache, starts, *(torch.empty(182, G * D, dtype=BF16, device="cuda") for _ in "kv"))
    got_q, out = torch.zeros_like(q), torch.zeros_like(q)
    kc, vc, k8, v8 = old
    where = (b.block_table, b.q_start, b.kv_len)
    sizes = (pr, b.num_pages, b.max_blocks, sr)
    A.attn_append_paged8(q, got_q, k, v, kc, vc, k8, v8, *where, b.rows, 4, H, G, D, G * D, H * D, H * D, G * D, G * D,
                         *sizes, q_weight=w, k_weight=w, rot_dim=D, table=table)
    A.attn_batch_paged8(got_q, kc, vc, k8, v8, out, *where, b.rows, 4, H, G, D, G * D, H * D, H * D, *sizes, D ** -0.5,
                        20, 3, 0.0, None, None, batch.workspace)
    k2, v2 = torch.empty_like(ks), torch.empty_like(vs)
    A.attn_read_paged8(kc, vc, k8, v8, k2, v2, b.block_table, starts, None, b.kv_len, 182, 4, G, D, G * D, G * D, G * D,
                       *sizes)
    assert A.attn_get_status() == 0
    assert torch.equal(want_q, got_q) and torch.equal(want, out) and torch.equal(ks, k2) and torch.equal(vs, v2)
    for a, c in zip((cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales), (kc, vc, k8, v8)):
        assert torch.equal(a, c)
    # First positions over 16 bits.
    pools = (b.k.nan_to_num(), b.v.nan_to_num())
    want = A.attend_paged(batch, q, *pools, window=20, sinks=3)
    A.attn_batch_paged_sinks(q, *pools, out.zero_(), *where, b.rows, 4, H, G, D, G * D, H * D, H * D, *sizes[:3],
                             D ** -0.5, 20, 0.0, None, None, batch.workspace, sinks=3)
    assert A.attn_get_status() == 0 and torch.equal(want, out)
    for call in (lambda: A.attn_batch_paged8(q, kc, vc, k8, v8, out, *where, b.rows, 4, H, G, D, G * D, H * D, H * D, pr,
                                             b.num_pages, b.max_blocks, 5, 0.1, 0, 0, 0.0, None, None, batch.workspace),
                 lambda: A.attn_read_paged8(kc, vc, k8, v8, k2, v2, b.block_table, starts, None, b.kv_len, 182, 4, G, D,
                                            G * D - 1, G * D, G * D, *sizes)):
        with pytest.raises(A.AttnError):
            call()
