"""Plain 64-bit forms of the 8-bit paged cache."""
import torch

from batch_ref import Batch


def exp_for(amax):
    """Smallest e from -14 to 7 with amax <= 448 * 2^e (64-bit tensor)."""
    e = torch.full_like(amax, -14.0)
    for x in range(-14, 7):
        e = torch.where(amax > 448.0 * 2.0 ** x, torch.full_like(e, x + 1.0), e)
    return e


def encode(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even, magnitudes above 448 to 448."""
    a = x.abs().clamp(2.0 ** -6, 2.0 ** 20)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3)
    return torch.where(x.isnan(), x, ((x / step).round() * step).clamp(-448.0, 448.0))


def decode(codes):
    return codes.view(torch.float8_e4m3fn).double()


class Batch8(Batch):
    """A ragged batch in shuffled pages of codes.  Pool rows that no sequence owns hold NaN codes, scales no range has."""

    def __init__(self, new, kv, H, G, D, page_rows, scale_rows, dtype=torch.bfloat16, seed=0, kv_dim=None, **more):
        super().__init__(new, kv, H, G, D, page_rows, dtype, seed=seed, kv_dim=kv_dim, **more)
        self.sr = scale_rows
        rows, w = self.k.shape
        g = torch.Generator(device="cuda").manual_seed(seed + 7)
        self.codes, self.scales = {}, {}
        owned = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for i, n in enumerate(kv):
            owned[self.slots(i, 0, n)] = True
        for name, x in (("k", self.k), ("v", self.v)):
            e = torch.randint(-3, 2, (rows // scale_rows, G), generator=g, device="cuda")
            c = torch.randn(rows, w, generator=g, device="cuda") * 0.8
            c = (c * 2.0 ** 3).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c[~owned] = 0x7f
            used = owned.view(-1, scale_rows).any(1)
            s = torch.where(used[:, None], e - 3 + 127, 255).to(torch.uint8)
            self.codes[name], self.scales[name] = c, s
            x[:, :G * D] = self.values(name, dtype)  # what the 16-bit cache of the same values holds
            x[~owned] = float("nan")

    def values(self, name, dtype=torch.float64):
        """Every pool row's values."""
        e = self.scales[name].double().clamp(127 - 14, 127 + 7) - 127
        e = e.repeat_interleave(self.sr, 0).repeat_interleave(self.D, 1)
        return (decode(self.codes[name][:, :self.G * self.D]) * torch.exp2(e)).to(dtype)

    def cache(self, A):
        return A.PagedCache8(self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"])

    def groups(self):
        """(sequence, first position, held, end) of every block of a scale that gets new rows."""
        out = []
        for i, (m, n) in enumerate(zip(self.new, self.kv)):
            for first in range((n - m) // self.sr * self.sr, n if m else 0, self.sr):
                out.append((i, first, max(0, n - m - first), min(self.sr, n - first)))
        return out


def attend64(b, q=None, window=0, sinks=0, softcap=0.0, slopes=None, prefix=None, scale=None):
    """(out, sum_j p_j |v_j|, largest |v| attended) in 64 bits from b.k and b.v; rows of no sequence are zeros."""
    q = b.q if q is None else q
    H, G, D = b.H, b.G, b.D
    gs = H // G
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape[0], H * D, dtype=torch.float64, device="cuda")
    mag, vmax = torch.zeros_like(out), 0.0
    for i, (n, length) in enumerate(zip(b.new, b.kv)):
        if n == 0 or length == 0:
            continue
        sl = b.slots(i, 0, length)
        k, v = (x[sl, :G * D].double().view(length, G, D) for x in (b.k, b.v))
        j = torch.arange(length, device="cuda")
        for r0 in range(0, n, 512):
            r1 = min(n, r0 + 512)
            p = torch.arange(length - n + r0, length - n + r1, device="cuda")[:, None]
            ok = j <= p
            if prefix is not None:
                ok = ok | (j < prefix[i])
            if window:
                ok = ok & ((j > p - window) | (j < sinks))
            used = ok.any(0).view(length, 1, 1)
            kk, vv = (torch.where(used, x, torch.zeros((), dtype=x.dtype, device="cuda")) for x in (k, v))
            x = q[b.starts[i] + r0:b.starts[i] + r1].double().view(r1 - r0, G, gs, D)
            s = scale * torch.einsum("nghd,jgd->ghnj", x, kk)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes.double().view(G, gs, 1, 1) * (p - j).abs()
            s = s.masked_fill(~ok, float("-inf"))
            w = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e300)).masked_fill(~ok, 0.0)
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
            rows = slice(b.starts[i] + r0, b.starts[i] + r1)
            out[rows] = torch.einsum("ghnj,jgd->nghd", w, vv).reshape(r1 - r0, H * D)
            mag[rows] = torch.einsum("ghnj,jgd->nghd", w, vv.abs()).reshape(r1 - r0, H * D)
            vmax = max(vmax, float(vv.abs().max()))
    return out, mag, vmax


def tolerance(ref, mag, vmax, dtype, p_dtype, keys):
    """Bound on |kernel - ref|, as attend_tolerance of batch_ref.py, for weights rounded to p_dtype and results to dtype."""
    sub = vmax * keys * 2.0 ** -25 if p_dtype == torch.float16 else 0.0
    half, half_p = torch.finfo(dtype).eps / 2, torch.finfo(p_dtype).eps / 2
    return 1.01 * (half_p * mag + half * ref.abs() + 2.0 ** -12 * mag) + sub + 1e-9
