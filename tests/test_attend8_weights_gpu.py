"""attn_batch_paged8 where values and weights are small: what the weights' rounding may cost, row by row and column by
column, against a plain 64-bit form.

Scores are within 2^-13 and weights within 2^-12 of themselves (attend_tolerance of batch_ref.py).  A weight is rounded to
fp16: by at most 2^-11 of itself and 2^-32 of the row's largest (single tokens: both times the key's V scale).  The result is
rounded once."""
import pytest
import torch

from cache8_ref import Batch8, decode

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16

BATCHES = {  # new, kv, H, G, D, page_rows, scale_rows; the single-token kernel?
    "tokens": (([1] * 6, [1, 5, 64, 300, 1000, 2049], 8, 2, 64, 16, 16), True),
    "tokens, heads of 128": (([1] * 4, [700, 129, 2000, 17], 16, 4, 128, 8, 4), True),
    "chunks": (([3, 130, 1, 64], [3, 1300, 700, 64], 8, 2, 64, 16, 8), False),
    "chunks, heads of 128": (([40, 7, 90], [1500, 500, 90], 12, 4, 128, 8, 1), False),
    "pairs": (([300, 257], [1400, 257], 8, 2, 128, 64, 16), False),
    "odd pages": (([1, 30, 9], [400, 900, 9], 8, 2, 64, 7, 7), False),
}


def bounds64(b, single, scale, v=None):
    """(out, bound on the kernel's error) in 64 bits, for rows of sequences; v: another pool of values."""
    H, G, D = b.H, b.G, b.D
    v = b.values("v") if v is None else v
    k = b.values("k")
    exps = torch.exp2(b.scales["v"].double().clamp(113, 134) - 127).repeat_interleave(b.sr, 0)
    out, tol = (torch.zeros(b.rows, H * D, dtype=torch.float64, device="cuda") for _ in range(2))
    half = torch.finfo(b.dtype).eps / 2
    for i, (n, length) in enumerate(zip(b.new, b.kv)):
        sl = b.slots(i, 0, length)
        kk, vv = (x[sl, :G * D].view(length, G, D) for x in (k, v))
        size = exps[sl]  # [length, G]
        p = torch.arange(length - n, length, device="cuda")[:, None]
        ok = torch.arange(length, device="cuda") <= p
        x = b.q[b.starts[i]:b.starts[i + 1]].double().view(n, G, H // G, D)
        s = scale * torch.einsum("nghd,jgd->ghnj", x, kk)
        w = torch.softmax(s.masked_fill(~ok, float("-inf")), -1)
        ref = torch.einsum("ghnj,jgd->nghd", w, vv)
        mag = torch.einsum("ghnj,jgd->nghd", w, vv.abs())
        seen = torch.einsum("nj,jgd->ngd", ok.double(), (vv.abs() / size[..., None]) if single else vv.abs())
        top = (w * size.T[:, None, None, :] if single else w).amax(-1).permute(2, 0, 1)  # [n, G, H / G]
        sub = 2.0 ** -32 * top[..., None] * seen[:, :, None, :]
        rows = slice(b.starts[i], b.starts[i + 1])
        out[rows] = ref.reshape(n, -1)
        tol[rows] = (1.01 * ((2.0 ** -11 + 2.0 ** -12) * mag + half * ref.abs()) + (1 + half) * sub).reshape(n, -1) + 2.0 ** -25
    return out, tol


def run(A, b, scale):
    out = A.attend_paged8(b.object(A), b.q, b.cache(A), scale=scale)
    assert A.attn_get_status() == 0
    return out.double()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("how", ["small", "a head of large ones", "each its own"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_values_of_small_scales(cuda_lib, name, how, dtype):
    """V's scales 2^-14 (and bytes below, which read as that), alone and with one kv head of 2^7; leaving the small values
    out, or taking a byte of 0 for a 32 times larger scale, would show."""
    A = cuda_lib
    sizes, single = BATCHES[name]
    b = Batch8(*sizes, dtype=dtype, seed=len(name))
    g = torch.Generator(device="cuda").manual_seed(2)
    choice = torch.tensor([0, 113, 114], dtype=torch.uint8, device="cuda")
    small = choice[torch.randint(0, 3, b.scales["v"].shape, generator=g, device="cuda")]
    if how == "a head of large ones":
        small[:, 0] = 134
    elif how == "each its own":
        small = torch.arange(b.G, device="cuda").mul(10).add(113).clamp(max=134).to(torch.uint8).expand_as(small).contiguous()
    b.scales["v"] = small
    scale = b.D ** -0.5
    ref, tol = bounds64(b, single, scale)
    got = run(A, b, scale)
    assert ((got - ref).abs() <= tol).all()
    v = b.values("v")
    low = (b.scales["v"] <= 114).repeat_interleave(b.sr, 0).repeat_interleave(b.D, 1)
    for wrong in (torch.where(low, 0.0, v), torch.where(low, 32 * v, v)):
        assert ((bounds64(b, single, scale, wrong)[0] - ref).abs() > 2 * tol).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("name", ["tokens", "tokens, heads of 128", "chunks, heads of 128", "pairs", "odd pages"])
def test_many_small_weights_beside_a_large_one(cuda_lib, name, dtype):
    """Keys of weight e^-18, 2^-26 of the largest, whose value is that of the result: fp16 would lose them all, were weights
    not made with 2^7 more."""
    A = cuda_lib
    sizes, single = BATCHES[name]
    b = Batch8(*sizes, dtype=dtype, seed=1)
    D = b.D
    b.q.fill_(1.0)
    for x in "kv":
        b.scales[x].fill_(127)
        b.codes[x].zero_()
    b.codes["v"].fill_(0x38)  # 1
    for i, (n, length) in enumerate(zip(b.new, b.kv)):  # the large ones: among the first keys that each kernel meets
        sl = b.slots(i, 0, length)[[0, length - n]]
        b.codes["k"][sl], b.codes["v"][sl] = 0x38, 0
    assert (decode(b.codes["k"]).unique() == torch.tensor([0.0, 1.0], device="cuda")).all()
    scale = 18.0 / D
    ref, tol = bounds64(b, single, scale)
    rows = [b.starts[i] + n - 1 for i, (n, length) in enumerate(zip(b.new, b.kv)) if length > 200]
    assert (ref[rows] > 5 * tol[rows]).all()
    assert ((run(A, b, scale) - ref).abs() <= tol).all()
