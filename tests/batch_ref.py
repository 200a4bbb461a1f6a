"""Plain 64-bit forms of the rotary, append and batched paged attention operators."""
import math

import torch


def theta(R, base=10000.0, scaling="none", factor=1.0, orig=0, fast=32.0, slow=1.0):
    out = []
    for i in range(R // 2):
        b = base * factor ** (R / (R - 2.0)) if scaling == "ntk" else base
        th = b ** (-2.0 * i / R)
        if scaling == "linear":
            th /= factor
        elif scaling == "by_parts":
            g = min(1.0, max(0.0, (orig * th / (2.0 * math.pi) - slow) / (fast - slow)))
            th *= g + (1.0 - g) / factor
        out.append(th)
    return torch.tensor(out, dtype=torch.float64)


def turn(x, pos, th, interleaved, m=1.0, sign=1.0):
    """x [rows, heads, D] (any type) turned in 64 bits by positions [rows]."""
    x = x.double().clone()
    R = 2 * th.numel()
    ang = pos.double()[:, None, None] * th.to(x.device)
    c, s = m * torch.cos(ang), sign * m * torch.sin(ang)
    ia, ib = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


class Batch:
    """A ragged batch in shuffled pages.  Every pool row that no sequence owns holds `junk`."""

    def __init__(self, new, kv, H, G, D, page_rows, dtype, seed=0, spare=2, junk=float("nan"), kv_dim=None, pad=0,
                 extra_blocks=1):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.H, self.G, self.D, self.pr, self.dtype = new, kv, H, G, D, page_rows, dtype
        n_blocks = [(n + page_rows - 1) // page_rows for n in kv]
        self.max_blocks = max(n_blocks) + extra_blocks
        self.num_pages = sum(n_blocks) + spare
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(kv), self.max_blocks), -1, dtype=torch.int32)
        at = 0
        for i, b in enumerate(n_blocks):
            self.table[i, :b] = order[at:at + b]
            at += b
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.starts, self.rows = starts, starts[-1] + pad
        w = G * D if kv_dim is None else kv_dim
        self.k = torch.full((self.num_pages * page_rows, w), junk, dtype=dtype, device="cuda")
        self.v = torch.full((self.num_pages * page_rows, w), junk, dtype=dtype, device="cuda")
        gd = torch.Generator(device="cuda").manual_seed(seed + 1)
        for i, n in enumerate(kv):
            sl = self.slots(i, 0, n)
            for x in (self.k, self.v):
                x[sl, :G * D] = torch.randn(n, G * D, generator=gd, device="cuda").to(dtype)
        self.q = torch.randn(self.rows, H * D, generator=gd, device="cuda").to(dtype)
        self.dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.q_start, self.kv_len, self.block_table = self.dev(starts), self.dev(kv), self.table.cuda()

    def slots(self, s, lo, hi):
        """Pool rows of positions [lo, hi) of sequence s."""
        t = torch.arange(lo, hi)
        return (self.table[s].long()[t // self.pr] * self.pr + t % self.pr).cuda()

    def object(self, A, block_table=None, q_start=None, kv_len=None):
        pick = lambda a, b: b if a is None else a  # noqa: E731
        return A.PagedBatch(pick(block_table, self.block_table), pick(q_start, self.q_start), pick(kv_len, self.kv_len),
                            self.H, self.G, self.D, self.pr)

    def attend(self, q=None, window=0, softcap=0.0, slopes=None, prefix=None, scale=None):
        """(out, sum_j p_j |v_j|, longest window) in 64 bits; rows of no sequence are zeros."""
        q = self.q if q is None else q
        H, G, D = self.H, self.G, self.D
        gs = H // G
        scale = 1.0 / math.sqrt(D) if scale is None else scale
        out = torch.zeros(q.shape[0], H * D, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(out)
        for i, (n, length) in enumerate(zip(self.new, self.kv)):
            if n == 0 or length == 0:
                continue
            sl = self.slots(i, 0, length)
            k = self.k[sl, :G * D].double().view(length, G, D).repeat_interleave(gs, 1)
            v = self.v[sl, :G * D].double().view(length, G, D).repeat_interleave(gs, 1)
            x = q[self.starts[i]:self.starts[i] + n].double().view(n, H, D)
            j = torch.arange(length, device="cuda")[None, :]
            p = torch.arange(length - n, length, device="cuda")[:, None]
            ok = j <= p
            if prefix is not None:
                ok = ok | (j < prefix[i])
            if window:
                ok = ok & (j > p - window)
            s = scale * torch.einsum("nhd,jhd->hnj", x, k)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes.double().view(H, 1, 1) * (p - j).abs()
            s = s.masked_fill(~ok, float("-inf"))
            w = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e300)).masked_fill(~ok, 0.0)
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
            # Values of keys that no row attends are left out, whatever they hold.
            used = ok.any(0)
            v = torch.where(used.view(length, 1, 1), v, torch.zeros((), dtype=v.dtype, device="cuda"))
            rows = slice(self.starts[i], self.starts[i] + n)
            out[rows] = torch.einsum("hnj,jhd->nhd", w, v).reshape(n, H * D)
            mag[rows] = torch.einsum("hnj,jhd->nhd", w, v.abs()).reshape(n, H * D)
        return out, mag


def attend_tolerance(ref, mag, dtype, keys):
    """Bound on |kernel - ref| for one output element.

    P is rounded to the cache's type: at most eps/2 of each weight, so eps/2
    sum p|v| in all; the result once more: eps/2 |ref|.  Scores are fp32: a dot
    product of 128 terms whose absolute sum (times scale) stays below 16 here is
    off by at most 128 * 2^-24 * 16 = 2^-13 in the score, a weight by that
    relatively, and the normalised weight by twice that, 2^-12.  fp16 weights
    below 2^-14 of the running reference lose at most 2^-25 each against a sum
    of at least 1: 2^-25 per key and unit of |v| (|v| < 6 for normal data)."""
    half = torch.finfo(dtype).eps / 2
    sub = 6.0 * keys * 2.0 ** -25 if dtype == torch.float16 else 0.0
    return 1.01 * (half * (mag + ref.abs()) + 2.0 ** -12 * mag) + sub + 1e-9
