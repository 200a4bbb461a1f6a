"""attn_rope_apply and attn_rope_table_scaled against plain 64-bit forms, and
the gradient against the transposed map and against differences."""
import pytest
import torch

from batch_ref import theta, turn

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
SCALES = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
          dict(scaling="by_parts", factor=4.0, orig_max_pos=2048, beta_fast=32.0, beta_slow=1.0)]


def ref_theta(R, kw):
    return theta(R, scaling=kw.get("scaling", "none"), factor=kw.get("factor", 1.0), orig=kw.get("orig_max_pos", 0),
                 fast=kw.get("beta_fast", 32.0), slow=kw.get("beta_slow", 1.0))


@pytest.mark.parametrize("R", [4, 16, 48, 128, 256])
@pytest.mark.parametrize("kw", SCALES)
def test_scaled_table(cuda_lib, kw, R):
    """fp32 entries of fp64 angles: half an fp32 step of entries below 1.4 (2^-24), plus the fp64 angle's own
    error at position 100000 (below 1e-9)."""
    m = 1.25 if kw else 1.0
    rows = 100001
    t = cuda_lib.rope_table(rows, R, 10000.0, scaling=kw.get("scaling", "none"), attn_factor=m,
                            **{k: v for k, v in kw.items() if k != "scaling"})
    pick = torch.tensor([0, 1, 2, 777, 4096, 65535, 100000])
    ang = pick.double()[:, None] * ref_theta(R, kw)
    got = t.cpu()[pick].double()
    assert (got[:, :R // 2] - m * torch.cos(ang)).abs().max() <= 1.25 * 2.0 ** -24 + 1e-9
    assert (got[:, R // 2:] - m * torch.sin(ang)).abs().max() <= 1.25 * 2.0 ** -24 + 1e-9


def test_unscaled_table_is_the_existing_one(cuda_lib):
    a = cuda_lib.rope_table(5000, 64, 10000.0)
    b = cuda_lib.rope_table(5000, 64, 10000.0, scaling="none")
    assert (a - b).abs().max() <= 2.0 ** -23  # two fp64 evaluations, each rounded to fp32


def tolerance(ref, x, dtype):
    """Table entries are off by 2^-24 m, the two products and their sum round in fp32 (2^-24 each): at most
    4 * 2^-24 * 2 max|x| m; then one rounding to the type."""
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    return half * ref.abs() + 8 * 1.5 * 2.0 ** -24 * (1 + half) * x.double().abs().max() + tiny


SHAPES = [  # rows, heads, D, R
    (1, 1, 64, 64), (7, 5, 128, 128), (33, 40, 128, 128), (300, 8, 80, 32), (19, 3, 96, 48), (64, 2, 50, 50),
    (5, 4, 33, 2), (129, 1, 8, 8), (17, 6, 256, 64), (3, 2, 1024, 1024), (40, 2, 64, 24), (1000, 12, 128, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,heads,D,R", SHAPES)
def test_forward_and_gradient(cuda_lib, rows, heads, D, R, dtype, interleaved):
    A = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    x = torch.randn(rows, heads * D, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 4096, (rows,), generator=g, device="cuda").to(torch.int32)
    kw = SCALES[(rows + D) % len(SCALES)] if R >= 4 else {}
    m = 1.2 if kw else 1.0
    table = A.rope_table(4096, R, 10000.0, scaling=kw.get("scaling", "none"), attn_factor=m,
                         **{k: v for k, v in kw.items() if k != "scaling"})
    th = ref_theta(R, kw)
    for call, sign in ((A.rope, 1.0), (A.rope_backward, -1.0)):
        y = call(x, table, heads, positions=pos, rot_dim=R, interleaved=interleaved)
        ref = turn(x.view(rows, heads, D), pos, th, interleaved, m, sign).view(rows, -1)
        assert ((y.double() - ref).abs() <= tolerance(ref, x, dtype)).all()
        back = torch.arange(heads * D, device="cuda") % D >= R
        assert torch.equal(y[:, back], x[:, back])
    assert A.attn_get_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_transpose_and_matches_differences(cuda_lib, interleaved):
    """<rope(x), dy> = <x, rope_backward(dy)>, and central differences of <rope(x), dy> in fp32: the map is
    linear, so a step of 2^6 leaves only rounding, 2 * 64 * 64 products of size ~1 at 2^-24 of the step."""
    A = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(3, 2 * 32, generator=g, device="cuda") for _ in range(2))
    pos = torch.tensor([3, 900, 17], dtype=torch.int32, device="cuda")
    table = A.rope_table(1000, 16, scaling="linear", factor=2.0, attn_factor=1.1)
    f = lambda t: (A.rope(t, table, 2, pos, 16, interleaved).double() * dy.double()).sum()  # noqa: E731
    dx = A.rope_backward(dy, table, 2, pos, 16, interleaved)
    assert abs(float(f(x)) - float((x.double() * dx.double()).sum())) <= 192 * 16 * 2.0 ** -24
    for r, c in ((0, 0), (1, 7), (1, 8), (1, 15), (2, 16), (2, 40), (0, 63)):
        d = torch.zeros_like(x)
        d[r, c] = 64.0
        diff = float((f(x + d) - f(x - d)) / 128.0)
        assert abs(diff - float(dx[r, c])) <= 32 * 2.0 ** -24 * 64


def test_rows_in_order_strided_views_in_place_and_other_streams(cuda_lib):
    A = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(2)
    base = torch.randn(50, 6 * 64 + 16, generator=g, device="cuda").bfloat16()
    keep = base.clone()
    table = A.rope_table(50, 64)
    want = A.rope(base[:, :4 * 64].contiguous(), table, 4)
    assert torch.equal(A.rope(base[:, :4 * 64], table, 4), want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    A.rope(base[:, :4 * 64], table, 4, out=base[:, :4 * 64], stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(base[:, :4 * 64], want) and torch.equal(base[:, 4 * 64:], keep[:, 4 * 64:])
    # Addresses and strides that do not allow 16-byte groups: the same values, one pair a thread.
    odd = torch.zeros(50, 4 * 64 + 3, device="cuda", dtype=torch.bfloat16)
    odd[:, 1:257] = keep[:, :256]
    assert torch.equal(A.rope(odd[:, 1:257], table, 4), want)


def test_position_past_the_table(cuda_lib):
    A = cuda_lib
    x = torch.ones(3, 2 * 16, device="cuda")
    table = A.rope_table(10, 8)
    y = A.rope(x, table, 2, positions=torch.tensor([9, 10, -1], dtype=torch.int32, device="cuda"), rot_dim=8)
    assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
    assert (y[1:].view(2, 2, 16)[..., :8] == 0).all() and (y.view(3, 2, 16)[..., 8:] == 1).all()
    assert (y[0].view(2, 16)[:, :8] != 0).all()


def test_no_rows(cuda_lib):
    x = torch.zeros(0, 128, device="cuda", dtype=torch.float16)
    assert cuda_lib.rope(x, cuda_lib.rope_table(4, 64), 2).shape == (0, 128)


def test_refusals(cuda_lib):
    A = cuda_lib
    x = torch.zeros(8, 128, device="cuda")
    table = A.rope_table(4, 64)
    with pytest.raises(A.AttnError):
        A.rope(x, table, 2)  # 8 rows in order, 4 in the table
    with pytest.raises(ValueError):
        A.rope(x, table.double(), 2, positions=torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        A.rope(x, table, 2, positions=torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        A.rope(x, table, 2, out=torch.zeros(8, 64, device="cuda"))
    with pytest.raises(ValueError):
        A.rope_table(4, 64, scaling="cubic")


@pytest.mark.parametrize("scaling", [None, "linear"])
def test_a_table_made_on_another_stream(cuda_lib, scaling):
    """Its memory belongs to that stream's order: what the current stream still does with memory that was freed there
    cannot reach it."""
    A = cuda_lib
    kw = {} if scaling is None else dict(scaling=scaling, factor=2.0)
    want = A.rope_table(4096, 128, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.empty_cache()
        for _ in range(4):
            junk = torch.empty(4096, 128, device="cuda")
            torch.cuda._sleep(2_000_000)
            junk.fill_(7.0)
            del junk
            got = A.rope_table(4096, 128, stream=stream, **kw)
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_a_table_without_a_scaling_carries_its_factor(cuda_lib):
    """attn_factor multiplies every entry, with or without a scaling: one rounding of a product with 1.5."""
    A = cuda_lib
    got, plain = A.rope_table(100, 64, attn_factor=1.5), A.rope_table(100, 64)
    assert ((got.double() - 1.5 * plain.double()).abs() <= 3 * 2.0 ** -24).all()
    assert torch.equal(got, A.rope_table(100, 64, scaling="none", attn_factor=1.5))


@pytest.mark.parametrize("D,R", [(64, 64), (80, 48), (33, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_position_past_the_table_writes_zeros_whatever_the_row_holds(cuda_lib, dtype, interleaved, D, R):
    """NaN and infinities among them; the columns behind the turned part pass."""
    A = cuda_lib
    table = A.rope_table(8, R)
    x = torch.ones(3, 2 * D, device="cuda", dtype=dtype)
    x[1, ::3], x[1, 1::3], x[1, 2::3] = float("nan"), float("inf"), float("-inf")
    pos = torch.tensor([7, 8, 0], dtype=torch.int32, device="cuda")
    for call in (A.rope, A.rope_backward):
        y = call(x, table, 2, positions=pos, rot_dim=R, interleaved=interleaved)
        assert A.attn_get_status() == A.ATTN_ERR_INVALID_ARG
        assert (y.view(3, 2, D)[1, :, :R] == 0).all()
        assert torch.equal(y.view(3, 2, D)[:, :, R:].isnan(), x.view(3, 2, D)[:, :, R:].isnan())
        assert torch.isfinite(y[[0, 2]].float()).all() and (y.view(3, 2, D)[[0, 2]][..., :R] != 0).any()
