"""attn_qk_norm_rope and its backward against plain 64-bit forms."""
import pytest
import torch

from batch_ref import theta, turn

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-6


def make(rows, heads, D, dtype, seed, pad=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = scale * torch.randn(rows, heads * D + pad, generator=g, device="cuda")
    return x.to(dtype)[:, :heads * D]


def forward64(x, w, D, pos, th, interleaved, eps=EPS, m=1.0):
    """(y, xh, r, z) of rows x [rows, heads*D]."""
    x = x.double().reshape(x.shape[0], -1, D)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    z = x * r * (1.0 if w is None else w.double())
    return turn(z, pos, th, interleaved, m), x * r, r, z


def backward64(x, dy, w, D, pos, th, interleaved, eps=EPS, m=1.0):
    """(dx, dw, bound on |dx| terms, sum of |dw| terms)."""
    _, xh, r, _ = forward64(x, w, D, pos, th, interleaved, eps, m)
    dz = turn(dy.double().reshape(xh.shape), pos, th, interleaved, m, -1.0)
    g = dz * (1.0 if w is None else w.double())
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    size = r * (g.abs().amax(-1, keepdim=True) + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    return dx, (dz * xh).sum((0, 1)), size, (dz * xh).abs().sum((0, 1))


def tiny(dtype):
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def check_forward(got, y, z, D, dtype):
    """The sum of D squares is off by at most D 2^-24 of itself, r by half of that and the rounding of rsqrt (2^-22);
    weight, table and turn add at most eight roundings.  A result is made of two values of z; it is rounded once."""
    rel = D * 2.0 ** -25 + 2.0 ** -22 + 8 * 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    tol = (1 + half) * rel * 2 * 1.5 * z.abs().amax(-1, keepdim=True) + half * y.abs() + tiny(dtype)
    assert ((got.double().reshape(y.shape) - y).abs() <= tol).all()


def check_backward(dx, dw, ref, D, dtype, w_dtype, terms):
    """As above for r and the turn; the mean of D products is off by D 2^-24 of the sum of their sizes.  dw is a sum of
    `terms` products in fp32, however they are grouped, each with the errors of its factors."""
    ref_dx, ref_dw, size, sum_dw = ref
    rel = D * 2.0 ** -23 + 2.0 ** -21 + 16 * 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    tol = (1 + half) * rel * 2 * size + half * ref_dx.abs() + tiny(dtype)
    assert ((dx.double().reshape(ref_dx.shape) - ref_dx).abs() <= tol).all()
    if dw is not None:
        half = torch.finfo(w_dtype).eps / 2
        # A turned dz is made of two values: allow for both in each product.
        tol = (rel + terms * 2.0 ** -24) * 2 * (sum_dw + sum_dw.mean()) + half * ref_dw.abs() + tiny(w_dtype)
        assert ((dw.double() - ref_dw).abs() <= tol).all()


SHAPES = [  # rows, H, G, D, R, interleaved
    (1, 1, 1, 2, 2, False), (3, 4, 2, 64, 64, False), (33, 14, 2, 64, 64, True), (130, 32, 8, 128, 128, False),
    (7, 3, 3, 80, 32, True), (65, 5, 1, 80, 32, False), (9, 2, 1, 50, 20, False), (5, 2, 2, 33, 6, True),
    (17, 6, 2, 128, 0, False), (11, 3, 1, 256, 128, False), (4, 2, 1, 255, 254, True), (2, 1, 1, 8, 8, True),
    (700, 8, 4, 96, 48, False), (1, 40, 1, 128, 64, False), (19, 2, 1, 256, 256, True), (6, 1, 3, 16, 16, False)]


@pytest.mark.parametrize("dtype,w_dtype", [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F32, BF16), (F16, None)])
@pytest.mark.parametrize("rows,H,G,D,R,interleaved", SHAPES)
def test_both_directions(cuda_lib, rows, H, G, D, R, interleaved, dtype, w_dtype):
    A = cuda_lib
    pad = 8 if D % 16 == 0 else 1
    q, k = make(rows, H, D, dtype, 1, pad), make(rows, G, D, dtype, 2, pad)
    dq, dk = make(rows, H, D, dtype, 3), make(rows, G, D, dtype, 4, pad)
    wq = wk = None
    if w_dtype is not None:
        wq, wk = (1 + 0.3 * make(1, 1, D, F32, s)[0].to(w_dtype) for s in (5, 6))
    pos = torch.randint(0, 500, (rows,), generator=torch.Generator().manual_seed(7)).to(torch.int32).cuda()
    table = A.rope_table(500, R, scaling="none") if R else None
    how = dict(table=table, positions=pos, rot_dim=R or None, interleaved=interleaved, eps=EPS)
    qo, ko = A.qk_norm_rope(q, k, H, G, wq, wk, **how)
    got = A.qk_norm_rope_backward(dq, dk, q, k, H, G, wq, wk, **how)
    assert A.attn_get_status() == 0
    th = theta(R)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        ref, _, _, z = forward64(x, w, D, pos, th, interleaved)
        check_forward(y, ref, z, D, dtype)
    for i, (x, dy, w, heads) in enumerate(((q, dq, wq, H), (k, dk, wk, G))):
        ref = backward64(x, dy, w, D, pos, th, interleaved)
        assert (got[2 + i] is None) == (w is None)
        check_backward(got[i], got[2 + i], ref, D, dtype, w_dtype, rows * heads)


@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (80, 32, True), (50, 20, False)])
def test_gradients_are_those_of_differences(cuda_lib, D, R, interleaved):
    """Along random directions: the 64-bit forward's central difference (step 1e-4: its error is below 1e-7 of the terms)."""
    A = cuda_lib
    rows, H, G = 6, 3, 2
    q, k, dq, dk = make(rows, H, D, F32, 1), make(rows, G, D, F32, 2), make(rows, H, D, F32, 3), make(rows, G, D, F32, 4)
    wq, wk = 1 + 0.3 * make(1, 1, D, F32, 5)[0], 1 + 0.3 * make(1, 1, D, F32, 6)[0]
    table, th = A.rope_table(rows, R), theta(R)
    pos = torch.arange(rows).cuda()
    got = A.qk_norm_rope_backward(dq, dk, q, k, H, G, wq, wk, table=table, rot_dim=R, interleaved=interleaved)
    for i, (x, dy, w) in enumerate(((q, dq, wq), (k, dk, wk))):
        ux, uw = make(rows, x.shape[1] // D, D, F32, 8).double(), make(1, 1, D, F32, 9)[0].double()

        def loss(t, s):
            return (forward64(x.double() + t * ux, w.double() + s * uw, D, pos, th, interleaved)[0].reshape(rows, -1) *
                    dy.double()).sum()

        h = 1e-4
        _, _, size, sum_dw = backward64(x, dy, w, D, pos, th, interleaved)
        slope = (loss(h, 0) - loss(-h, 0)) / (2 * h)
        assert abs(slope - (got[i].double() * ux).sum()) <= 1e-5 * (size.reshape(rows, -1) * ux.abs()).sum()
        slope = (loss(0, h) - loss(0, -h)) / (2 * h)
        assert abs(slope - (got[2 + i].double() * uw).sum()) <= 1e-5 * (sum_dw * uw.abs()).sum()


def test_rows_without_positions_a_scaled_table_and_places(cuda_lib):
    """Row t at position t, the table's factor in both directions, results in place of their inputs."""
    A = cuda_lib
    rows, H, G, D = 40, 4, 2, 64
    table = A.rope_table(64, D, scaling="linear", factor=2.0, attn_factor=1.5)
    th = theta(D, scaling="linear", factor=2.0)
    pos = torch.arange(rows).cuda()
    for dtype, pad in ((F32, 0), (BF16, 8), (F16, 3)):
        q, k = make(rows, H, D, dtype, 1, pad), make(rows, G, D, dtype, 2, pad)
        dq, dk = make(rows, H, D, dtype, 3, pad), make(rows, G, D, dtype, 4, pad)
        w = 1 + 0.3 * make(1, 1, D, dtype, 5)[0]
        apart = A.qk_norm_rope(q, k, H, G, w, None, table=table)
        ref, _, _, z = forward64(q, w, D, pos, th, False, m=1.5)
        check_forward(apart[0], ref, z, D, dtype)
        grads = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, None, table=table)
        check_backward(grads[0], grads[2], backward64(q, dq, w, D, pos, th, False, m=1.5), D, dtype, dtype, rows * H)
        # (The same rows again, equally far apart: other strides may take other sums.)
        q2, k2 = make(rows, H, D, dtype, 1, pad), make(rows, G, D, dtype, 2, pad)
        dq2, dk2 = make(rows, H, D, dtype, 3, pad), make(rows, G, D, dtype, 4, pad)
        again = A.qk_norm_rope_backward(dq2, dk2, q2, k2, H, G, w, None, table=table, dq_out=dq2, dk_out=k2)
        assert torch.equal(dq2, grads[0]) and torch.equal(k2, grads[1]) and torch.equal(again[2], grads[2])
        k2 = make(rows, G, D, dtype, 2, pad)
        A.qk_norm_rope(q2, k2, H, G, w, None, table=table, q_out=q2, k_out=k2)
        assert torch.equal(q2, apart[0]) and torch.equal(k2, apart[1])


def test_large_batches_and_repeated_calls(cuda_lib):
    """More rows than one round of blocks; the same bits every time."""
    A = cuda_lib
    rows, H, G, D = 5003, 8, 2, 128
    q, k, dq, dk = (make(rows, h, D, BF16, i) for i, h in enumerate((H, G, H, G)))
    w = 1 + 0.3 * make(1, 1, D, F32, 5)[0]
    table = A.rope_table(rows, D)
    a = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table)
    b = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    pos = torch.arange(rows).cuda()
    for i, (x, dy, h) in enumerate(((q, dq, H), (k, dk, G))):
        # (Sums of a few hundred terms a lane, joined in a tree.)
        check_backward(a[i], a[2 + i], backward64(x, dy, w, D, pos, theta(D), False), D, BF16, F32, 512)


def test_zero_rows_extreme_values_and_positions_past_the_table(cuda_lib):
    A = cuda_lib
    H, G, D = 2, 1, 64
    w = torch.ones(D, device="cuda")
    table = A.rope_table(8, D)
    e = torch.empty(0, H * D, device="cuda"), torch.empty(0, G * D, device="cuda")
    assert A.qk_norm_rope(*e, H, G, w, w, table=table)[0].shape == (0, H * D)
    grads = A.qk_norm_rope_backward(*e, *e, H, G, w, w, table=table)
    assert (grads[2] == 0).all() and (grads[3] == 0).all()
    # Heads of zeros stay zeros; tiny and large ones are as the formula has them.
    q, k = make(4, H, D, F32, 1), make(4, G, D, F32, 2)
    q[0] = 0
    q[1] *= 1e-12
    q[2] *= 1e15
    qo, _ = A.qk_norm_rope(q, k, H, G, w, w, table=table)
    ref, _, _, z = forward64(q, w, D, torch.arange(4).cuda(), theta(D), False)
    check_forward(qo, ref, z, D, F32)
    assert A.attn_get_status() == 0
    # A NaN or an infinity stays within its head.
    q[3, 5], q[2, D + 1] = float("nan"), float("inf")
    again, _ = A.qk_norm_rope(q, k, H, G, w, w, table=table)
    assert again[3, :D].isnan().all() and torch.equal(again[3, D:], qo[3, D:]) and torch.equal(again[2, :D], qo[2, :D])
    # Past the table: zeros in the turned columns, NaN or not.
    for R, interleaved in ((64, False), (32, True), (20, False)):
        pos = torch.tensor([0, 8, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
        q2 = make(4, H, D, F32, 1)
        q2[1, 0] = float("nan")
        part = A.rope_table(8, R)
        qo, ko = A.qk_norm_rope(q2, k, H, G, w, w, table=part, positions=pos, rot_dim=R, interleaved=interleaved)
        assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
        turned = qo.view(4, H, D)[..., :R]
        assert (turned[1:3] == 0).all() and (turned[[0, 3]] != 0).any(-1).all() and (ko.view(4, G, D)[1, :, :R] == 0).all()
        dq, dk = make(4, H, D, F32, 3), make(4, G, D, F32, 4)
        grads = A.qk_norm_rope_backward(dq, dk, q2, k, H, G, w, w, table=part, positions=pos, rot_dim=R,
                                        interleaved=interleaved)
        assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
        cut = dk.clone().view(4, G, D)
        cut[1:3, :, :R] = 0
        ref = backward64(k, cut.reshape(4, -1), w, D, pos * (pos < 8), theta(R), interleaved)
        check_backward(grads[1], grads[3], ref, D, F32, F32, 4)


def test_streams_and_graphs(cuda_lib):
    A = cuda_lib
    rows, H, G, D = 300, 4, 2, 128
    q, k, dq, dk = (make(rows, h, D, F16, i) for i, h in enumerate((H, G, H, G)))
    w = 1 + 0.3 * make(1, 1, D, F16, 5)[0]
    table = A.rope_table(rows, D)
    want = A.qk_norm_rope(q, k, H, G, w, w, table=table)
    grads = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = A.qk_norm_rope(q, k, H, G, w, w, table=table, stream=side)
    back = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + grads, got + back))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = A.qk_norm_rope(q, k, H, G, w, w, table=table)
        back = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table)
    for x in got + back:
        x.zero_()
    q.mul_(0.5)  # (a norm does not see it, but for eps)
    dq.mul_(2)
    graph.replay()
    want = A.qk_norm_rope(q, k, H, G, w, w, table=table)
    grads = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, table=table)
    assert all(torch.equal(a, b) for a, b in zip(want + grads, got + back))


@pytest.mark.parametrize("H,G,D,interleaved", [(5, 3, 128, False), (7, 1, 64, False), (3, 5, 80, True), (5, 2, 36, False)])
def test_an_infinite_gradient_reaches_its_own_column_of_the_weights(cuda_lib, H, G, D, interleaved):
    """Heads that do not fill a warp: the lanes that are left add nothing, not a product of zero and infinity."""
    A = cuda_lib
    w = torch.ones(D, device="cuda")
    q, k, dq, dk = (make(3, n, D, F32, seed) for n, seed in ((H, 1), (G, 2), (H, 3), (G, 4)))
    dq[2, (H - 1) * D + 9] = dk[1, (G - 1) * D + 3] = float("inf")
    _, _, dwq, dwk = A.qk_norm_rope_backward(dq, dk, q, k, H, G, w, w, interleaved=interleaved)
    for dw, at, x in ((dwq, 9, q[2, (H - 1) * D + 9]), (dwk, 3, k[1, (G - 1) * D + 3])):
        assert dw[at] == float("inf") * torch.sign(x)
        assert dw.isfinite().sum() >= D - 2  # (and the column that it would turn with)


def same_values(got, ref, tol):
    """NaN where ref is, the same infinities, and finite values within tol."""
    assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.isinf(), ref.isinf())
    assert torch.equal(got[ref.isinf()].double(), ref[ref.isinf()])
    fine = ref.isfinite()
    assert ((got.double() - ref).abs() <= tol)[fine].all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D,R,interleaved", [(128, 0, False), (128, 0, True), (64, 32, False), (64, 32, True),
                                             (80, 32, True), (96, 48, False), (36, 10, True)])
def test_infinities_stay_in_columns_that_do_not_turn(cuda_lib, D, R, interleaved, dtype):
    """A column behind rot_dim (or any, without a turn) meets no other one, but through its head's sums."""
    A = cuda_lib
    rows, H, G = 4, 3, 2
    table = A.rope_table(rows, R) if R else None
    th, pos = theta(R), torch.arange(rows).cuda()
    how = dict(table=table, rot_dim=R or None, interleaved=interleaved)
    w = 1 + 0.3 * make(1, 1, D, F32, 5)[0]
    q, k, dq, dk = (make(rows, n, D, dtype, seed) for n, seed in ((H, 1), (G, 2), (H, 3), (G, 4)))
    half = torch.finfo(dtype).eps / 2
    for at in (R, R + 9, D - 2):
        y, u = dq.clone(), dk.clone()
        y[1, D + at], u[2, D + at] = float("inf"), -float("inf")
        got = A.qk_norm_rope_backward(y, u, q, k, H, G, w, w, **how)
        for i, (x, dy) in enumerate(((q, y), (k, u))):
            dx, dw, _, _ = backward64(x, dy, w, D, pos, th, interleaved)
            assert dw.isinf().sum() == 1 and dw.isnan().sum() == 0
            # (Finite values: those of test_both_directions.  Here a coarse bound will do.)
            same_values(got[i].view(dx.shape), dx, 2 * half * dx.abs() + 1e-4)
            same_values(got[2 + i], dw, 1e-4)
        x = q.clone()
        x[1, D + at] = float("inf")
        got = A.qk_norm_rope(x, k, H, G, w, w, **how)[0]
        ref = forward64(x, w, D, pos, th, interleaved)[0]
        assert ref.isnan().sum() == 1
        same_values(got.view(ref.shape), ref, 2 * half * ref.abs() + 1e-4)
    assert A.attn_get_status() == 0
