"""Cases of the operators around an 8-bit paged cache: norms of query and key
heads with their rotary turn, a cache quantised as it is written and read
back, attention over it, and attention with a sliding window and first tokens
that stay visible.

Each operator stands here in plain torch operations (32 bits, rounded once at
the end) and as the calls of this package that replace them; `own` picks which
of the two `run` makes.  `exact` gives the same results from the definitions
in 64 bits.

    norm      z = w x / sqrt(mean(x^2) + eps) over the D columns of each head of Q and K, then pairs
              (i, i + R/2), or (2i, 2i + 1), of its first R columns turn by the angle p theta_i; the
              gradients of x and w
    append8   position t of a sequence is row t % page_rows of its page; a block of scale_rows rows and
              a kv head share a scale 2^e, the smallest with max|x| <= 448 2^e (e from -14 to 7) over the
              block's rows written so far.  Codes are x 2^-e rounded to e4m3; rows that a block held
              before are rounded again where its scale grows
    read8     the values that a range of each sequence's positions stands for
    attend8   the row at position p attends [0, min(sinks, hi)) and [max(0, p + 1 - window), hi) with
              hi = max(p + 1, min(prefix, kv_len)) and score cap * tanh(scale q.k / cap) - slope_h |p - j|
    attend    the same over a 16-bit cache
"""
import math
import random

import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_ESIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
_BASE, _EPS = 10000.0, 1e-6


# ------------------------------------------------------------------ cases
def listed():
    """Twelve cases.  32 query heads over 8 kv heads of 128 columns are the
    repository's benchmark heads; 16384 its decode cache, 8192 its forward."""
    return [
        # Q and K heads of a packed projection, a training or prompt step of a model that norms each head.
        _norm("norm_prompt_bf16", rows=8192, H=32, G=8, D=128, R=128, stride=6144),
        # One token of each of a batch of sequences: latency.
        _norm("norm_step_fp16", rows=33, H=14, G=2, D=64, R=64, stride=1152, dtype="fp16", pos_max=16384),
        # The gradient of the first.
        _norm("norm_grad_bf16", rows=8192, H=32, G=8, D=128, R=128, stride=6144, grad=True),
        # The gradient in fp32 at odd sizes, heads turned in part, interleaved.
        _norm("norm_grad_fp32_part", rows=4099, H=8, G=4, D=80, R=32, stride=1280, dtype="fp32", interleaved=True,
              grad=True, pos_max=16384),
        # A serving step: one token of 64 sequences, K and Q normed and turned on the way.
        _append("append8_step_bf16", n_seqs=64, new=(1, 1), ctx=(1, 2047), page_rows=16, scale_rows=16, norm=True),
        # Chunks of prompts behind ragged contexts.
        _append("append8_chunks_bf16", n_seqs=4, new=(1500, 2048), ctx=(0, 511), page_rows=64, scale_rows=32),
        # Whole sequences read back, for a computation that takes 16-bit rows.
        _read("read8_prefixes_bf16", n_seqs=17, kv=(1, 8192), page_rows=64, scale_rows=64),
        # A few short ones, a scale for every token, odd heads.
        _read("read8_short_fp32", n_seqs=3, kv=(20, 90), page_rows=24, scale_rows=1, dtype="fp32", G=3, D=80),
        # A serving step of 64 sequences of very different lengths in small pages.
        _attend("attend8_tokens_bf16", n_seqs=64, new=(1, 1), ctx=(0, 16383), page_rows=16, bits=8),
        # A chunk of each of two prompts behind long caches.
        _attend("attend8_chunks_bf16", n_seqs=2, new=(512, 512), ctx=(16384, 32000), page_rows=64, bits=8),
        # Single tokens of long chats that keep a window and their first tokens, seven query heads a kv head.
        _attend("sinks_tokens_fp16", n_seqs=33, new=(1, 1), ctx=(100, 16000), page_rows=32, bits=16, dtype="fp16",
                H=14, G=2, D=64, window=4096, sinks=4),
        # A whole prompt of a model with such layers.
        _attend("sinks_prompt_bf16", n_seqs=1, new=(8192, 8192), ctx=(0, 0), page_rows=64, bits=16, window=2048,
                sinks=128),
    ]


def _named(name, c):
    return dict(c, name=name) if name else c


def _norm(name, rows, H, G, D, R, stride, dtype="bf16", interleaved=False, grad=False, pos_max=None):
    return _named(name, dict(op="norm", rows=rows, H=H, G=G, D=D, R=R, stride=stride, dtype=dtype,
                             interleaved=interleaved, grad=grad, pos_max=pos_max or rows))


def _append(name, n_seqs, new, ctx, page_rows, scale_rows, src="bf16", H=32, G=8, D=128, R=None, interleaved=False,
            norm=False, ragged=1):
    return _named(name, dict(op="append8", n_seqs=n_seqs, new_min=new[0], new_max=new[1], ctx_min=ctx[0],
                             ctx_max=ctx[1], page_rows=page_rows, scale_rows=scale_rows, src=src, H=H, G=G, D=D,
                             R=D if R is None else R, interleaved=interleaved, norm=norm, ragged=ragged))


def _read(name, n_seqs, kv, page_rows, scale_rows, dtype="bf16", G=8, D=128, first=False, ragged=3):
    return _named(name, dict(op="read8", n_seqs=n_seqs, new_min=0, new_max=0, ctx_min=kv[0], ctx_max=kv[1],
                             page_rows=page_rows, scale_rows=scale_rows, dtype=dtype, H=G, G=G, D=D, first=first,
                             ragged=ragged))


def _attend(name, n_seqs, new, ctx, page_rows, bits, dtype="bf16", scale_rows=None, H=32, G=8, D=128, softcap=0.0,
            window=0, sinks=0, alibi=False, prefix=False, ragged=2):
    return _named(name, dict(op="attend", n_seqs=n_seqs, new_min=new[0], new_max=new[1], ctx_min=ctx[0],
                             ctx_max=ctx[1], page_rows=page_rows, bits=bits, scale_rows=scale_rows or page_rows,
                             dtype=dtype, H=H, G=G, D=D, softcap=softcap, window=window, sinks=sinks, alibi=alibi,
                             prefix=prefix, ragged=ragged))


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _divisor(rng, n):
    return rng.choice([d for d in range(1, n + 1) if n % d == 0])


def draw(rng):
    big = {c["name"]: work(c) for c in listed()}
    while True:
        op = rng.choice(["norm", "append8", "read8", "attend", "attend", "attend"])
        ragged = rng.randrange(1 << 30)
        interleaved = rng.random() < 0.4
        page_rows = rng.choice([16, 32, 64, 128, 8 * rng.randrange(1, 20)])
        if op == "norm":
            D = rng.choice([64, 128, 80, 96, 50, rng.randrange(8, 129, 2)])
            R = max(2, rng.choice([D, D // 4 * 2, rng.randrange(2, D + 1, 2)]))
            G = rng.choice([1, 2, 3, 4, 8])
            H = G * rng.choice([1, 2, 4, 5])
            rows = _log(rng, 1, 16384)
            c = _norm(None, rows, H, G, D, R, (H + G) * D + rng.choice([0, 8, 1, D]),
                      rng.choice(["bf16", "fp16", "fp32"]), interleaved, rng.random() < 0.5,
                      max(rows, _log(rng, 64, 131072)))
            if work(c)["bytes"] <= big["norm_grad_bf16"]["bytes"]:
                return c
        elif op == "append8":
            D = rng.choice([64, 128, 96, 80, 48])
            G = rng.choice([1, 2, 3, 4, 8])
            c = _append(None, _log(rng, 1, 128), (1, rng.choice([1, _log(rng, 1, 2048)])), (0, _log(rng, 1, 2048)),
                        page_rows, _divisor(rng, page_rows), rng.choice(["bf16", "fp16", "fp32"]),
                        G * rng.choice([0, 1, 2, 4, 5, 8]), G, D, rng.choice([D, D // 2, D // 4]), interleaved,
                        rng.random() < 0.5, ragged)
            if work(c)["bytes"] <= big["append8_chunks_bf16"]["bytes"]:
                return c
        elif op == "read8":
            c = _read(None, _log(rng, 1, 64), (1, _log(rng, 1, 8192)), page_rows, _divisor(rng, page_rows),
                      rng.choice(["bf16", "fp16", "fp32"]), rng.choice([1, 2, 3, 4, 8]),
                      rng.choice([64, 128, 96, 80, 48]), rng.random() < 0.5, ragged)
            if work(c)["bytes"] <= big["read8_prefixes_bf16"]["bytes"]:
                return c
        else:
            G = rng.choice([1, 2, 4, 8])
            bits = rng.choice([8, 8, 16])
            window = rng.choice([0, _log(rng, 1, 8192)]) if bits == 8 else _log(rng, 1, 8192)
            c = _attend(None, _log(rng, 1, 96), (1, rng.choice([1, 1, _log(rng, 1, 2048)])), (0, _log(rng, 1, 32768)),
                        page_rows, bits, rng.choice(["bf16", "fp16"]), _divisor(rng, page_rows),
                        G * rng.choice([1, 2, 4, 8, 3, 7, 16]), G, rng.choice([64, 128, 128, 64, 96, 80]),
                        rng.choice([0.0, 0.0, 30.0, 50.0]), window, rng.choice([1, 4, _log(rng, 1, 300)]) if window else 0,
                        rng.random() < 0.3, rng.random() < 0.25, ragged)
            w = work(c)
            if w["flops"] <= big["attend8_chunks_bf16"]["flops"] and w["bytes"] <= big["attend8_tokens_bf16"]["bytes"]:
                return c


def _lengths(case):
    """New rows, total length and prefix of each sequence, spread over their ranges."""
    rng = random.Random(case["ragged"])
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["n_seqs"])]
    kv = [n + rng.randint(case["ctx_min"], case["ctx_max"]) for n in new]
    prefix = [rng.randint(0, n) for n in kv]
    return new, kv, prefix


def _keys_of(case, p, kv, prefix):
    """(end of the first tokens, lo, hi): the row at position p attends [0, end) and [lo, hi)."""
    hi = max(p + 1, min(prefix, kv)) if case["prefix"] else p + 1
    lo = max(0, p + 1 - case["window"]) if case["window"] else 0
    return min(case["sinks"], lo), lo, hi


def work(case):
    D, H, G = case["D"], case["H"], case["G"]
    if case["op"] == "norm":
        heads = case["rows"] * (H + G)
        x = heads * D * _ESIZE[case["dtype"]]
        table = min(case["rows"], case["pos_max"]) * case["R"] * 4 + 4 * case["rows"]
        if case["grad"]:
            return {"bytes": 3 * x + table, "flops": heads * (12 * D + 3 * case["R"])}
        return {"bytes": 2 * x + table, "flops": heads * (5 * D + 3 * case["R"])}
    new, kv, prefix = _lengths(case)
    rows = sum(new)
    if case["op"] == "append8":
        es = _ESIZE[case["src"]]
        blocks = sum((n - 1) // case["scale_rows"] + 1 for n in new)
        return {"bytes": rows * (2 * G * D * (es + 1) + H * D * (es + min(es, 2)) + case["R"] * 4) + 2 * blocks * G,
                "flops": rows * (G + H) * (3 * case["R"] + (5 * D if case["norm"] else 0)) + 4 * rows * G * D}
    if case["op"] == "read8":
        n = sum(b - a for a, b in zip(_firsts(case, kv), kv))
        return {"bytes": 2 * n * G * D * (1 + _ESIZE[case["dtype"]]) + 2 * n * G // case["scale_rows"],
                "flops": 2 * n * G * D}
    pairs = keys = 0
    for n, length, pre in zip(new, kv, prefix):
        first, last, sink = length, 0, 0
        for p in range(length - n, length):
            end, lo, hi = _keys_of(case, p, length, pre)
            pairs += hi - lo + end
            first, last, sink = min(first, lo), max(last, hi), max(sink, end)
        keys += last - first + min(sink, first)
    cache = D if case["bits"] == 16 else D / 2
    scales = 0 if case["bits"] == 16 else 2 * keys * G // case["scale_rows"]
    return {"bytes": int(4 * keys * G * cache) + scales + 4 * rows * H * D, "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ inputs
def _theta(R):
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    return _BASE ** (-2.0 * i / R)


def _table(max_pos, R):
    """[max_pos, R]: cos of the R/2 pair angles of each position, then their sin."""
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * _theta(R)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _firsts(case, kv):
    """First position that is read of each sequence."""
    rng = random.Random(case["ragged"] + 1)
    return [rng.randint(0, n - 1) if case["first"] else 0 for n in kv]


def _exponents(amax):
    """Smallest e in -14 .. 7 with amax <= 448 2^e = 0.875 2^(e + 9)."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875), -14).clamp(-14, 7)


def _pool8(g, rows, G, D, scale_rows):
    """Codes and scale bytes of a cache whose heads and blocks differ in size."""
    codes = torch.empty(rows, G * D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows // scale_rows, G, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (G * D * scale_rows)) * scale_rows
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = torch.empty(b - a, G, D, device="cuda").normal_(generator=g)
        x = x.view(-1, scale_rows, G, D)
        size = torch.empty(x.shape[0], 1, G, 1, device="cuda").uniform_(-0.7, 0.7, generator=g)
        x = x * torch.exp2(size)
        e = _exponents(x.abs().amax((1, 3)))
        y = x * torch.exp2(-e.float())[:, None, :, None]
        codes[a:b] = y.reshape(b - a, G * D).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[a // scale_rows:b // scale_rows] = (e + 127).to(torch.uint8)
    return codes, scales


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)

    s = {"case": case}
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "norm":
        dt = _DT[case["dtype"]]
        base = randn(case["rows"], case["stride"], dtype=dt)
        s["q"], s["k"] = base[:, :H * D], base[:, H * D:(H + G) * D]
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * randn(D, dtype=torch.float32)).to(dt), \
            (1.0 + 0.2 * randn(D, dtype=torch.float32)).to(dt)
        pos = torch.randint(0, case["pos_max"], (case["rows"],), generator=g, device="cuda")
        if case["pos_max"] == case["rows"]:
            pos = torch.arange(case["rows"], device="cuda")  # a prompt from its first token
        s["pos"] = pos.to(torch.int32)
        if case["grad"]:
            s["dq"], s["dk"] = randn(case["rows"], H * D, dtype=dt), randn(case["rows"], G * D, dtype=dt)
        return s
    new, kv, prefix = _lengths(case)
    pr, kv_dim = case["page_rows"], G * D
    blocks = [(n + pr - 1) // pr for n in kv]
    num_pages = sum(blocks) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(kv), max(blocks)), -1, dtype=torch.int32)  # entries past a sequence's pages name none
    at = 0
    for i, b in enumerate(blocks):
        table[i, :b] = order[at:at + b]
        at += b
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    if case["op"] != "attend" or case["bits"] == 8:
        s["k_pages"], s["k_scales"] = _pool8(g, num_pages * pr, G, D, case["scale_rows"])
        s["v_pages"], s["v_scales"] = _pool8(g, num_pages * pr, G, D, case["scale_rows"])
    else:
        s["k_pages"] = randn(num_pages * pr, kv_dim, dtype=_DT[case["dtype"]])
        s["v_pages"] = randn(num_pages * pr, kv_dim, dtype=_DT[case["dtype"]])
    s["block_table"] = table.cuda()
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["new"], s["kv"], s["prefix"], s["num_pages"] = new, kv, prefix, num_pages
    if case["op"] == "append8":
        src = _DT[case["src"]]
        s["k_new"], s["v_new"] = randn(rows, kv_dim, dtype=src), randn(rows, kv_dim, dtype=src)
        s["q"] = randn(rows, H * D, dtype=src) if H else None
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (1.0 + 0.2 * randn(D, dtype=torch.float32)).to(src), \
                (1.0 + 0.2 * randn(D, dtype=torch.float32)).to(src)
            s["q_weight"] = s["q_weight"] if H else None
    elif case["op"] == "read8":
        s["first"] = _firsts(case, kv)
        starts = [0]
        for a, b in zip(s["first"], kv):
            starts.append(starts[-1] + b - a)
        s["total"] = starts[-1]
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["first_pos"] = torch.tensor(s["first"], dtype=torch.int32, device="cuda")
    else:
        s["q"] = randn(rows, H * D, dtype=_DT[case["dtype"]])
        if case["alibi"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
        if case["prefix"]:
            s["prefix_len"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "norm":
        s["table"] = _table(case["pos_max"], case["R"])
        s["q_out"] = torch.empty(case["rows"], H * D, dtype=s["q"].dtype, device="cuda")
        s["k_out"] = torch.empty(case["rows"], G * D, dtype=s["q"].dtype, device="cuda")
        return s
    if case["op"] == "append8":
        s["table"] = _table(max(s["kv"]), case["R"])
        if H:
            out = torch.bfloat16 if case["src"] == "fp32" else _DT[case["src"]]
            s["q_out"] = torch.empty(s["q"].shape, dtype=out, device="cuda")
    elif case["op"] == "read8":
        s["k_out"], s["v_out"] = (torch.empty(s["total"], G * D, dtype=_DT[case["dtype"]], device="cuda")
                                  for _ in range(2))
    else:
        s["out"] = torch.empty_like(s["q"])
    if own:
        import attention_gqa_online_gb300 as A
        s["batch"] = A.PagedBatch(s["block_table"], s["q_start"], s["kv_len"], max(H, G), G, D, case["page_rows"])
        if "k_scales" in s:
            s["cache"] = A.PagedCache8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _RUN_OWN[case["op"]](state, case)
    return _RUN_PLAIN[case["op"]](state, case)


def _own_norm(s, case):
    import attention_gqa_online_gb300 as A
    how = dict(positions=s["pos"], rot_dim=case["R"], interleaved=case["interleaved"], eps=_EPS)
    if not case["grad"]:
        A.qk_norm_rope(s["q"], s["k"], case["H"], case["G"], s["q_weight"], s["k_weight"], table=s["table"],
                       q_out=s["q_out"], k_out=s["k_out"], **how)
        return {"q": s["q_out"], "k": s["k_out"]}
    dq, dk, dwq, dwk = A.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], case["H"], case["G"], s["q_weight"],
                                               s["k_weight"], table=s["table"], dq_out=s["q_out"], dk_out=s["k_out"],
                                               **how)
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def _state8(s):
    """The cache as the values that it is made of."""
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"k_pages": s["k_pages"].view(e4), "v_pages": s["v_pages"].view(e4), "k_scales": s["k_scales"].view(e8),
            "v_scales": s["v_scales"].view(e8)}


def _own_append(s, case):
    import attention_gqa_online_gb300 as A
    A.append_paged8(s["batch"], s["k_new"], s["v_new"], s["cache"], q=s["q"], q_out=s.get("q_out"), table=s["table"],
                    rot_dim=case["R"], interleaved=case["interleaved"], q_weight=s["q_weight"],
                    k_weight=s["k_weight"], eps=_EPS)
    out = _state8(s)
    if case["H"]:
        out["q"] = s["q_out"]
    return out


def _own_read(s, case):
    import attention_gqa_online_gb300 as A
    A.read_paged8(s["batch"], s["cache"], s["starts"], s["k_out"], s["v_out"], first=s["first_pos"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attend(s, case):
    import attention_gqa_online_gb300 as A
    how = dict(out=s["out"], window=case["window"], sinks=case["sinks"], softcap=case["softcap"],
               alibi_slopes=s.get("slopes"), prefix_len=s.get("prefix_len"))
    if case["bits"] == 8:
        return A.attend_paged8(s["batch"], s["q"], s["cache"], **how)
    return A.attend_paged(s["batch"], s["q"], s["k_pages"], s["v_pages"], **how)


_RUN_OWN = {"norm": _own_norm, "append8": _own_append, "read8": _own_read, "attend": _own_attend}


def _turn(x, table_rows, R, interleaved, sign):
    """x [rows, heads, D] in 32 bits, turned by each row's table entries."""
    cos, sin = table_rows[:, None, :R // 2], sign * table_rows[:, None, R // 2:]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _unit(x):
    """(x / rms, 1 / rms) over the last axis."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    return x * r, r


def _plain_norm(s, case):
    rows, D, out = case["rows"], case["D"], {}
    tab = s["table"][s["pos"].long()]
    for name in ("q", "k"):
        x = s[name].float().reshape(rows, -1, D)
        w = s[name + "_weight"].float()
        n, r = _unit(x)
        if not case["grad"]:
            out[name] = _turn(n * w, tab, case["R"], case["interleaved"], 1.0).reshape(rows, -1).to(s[name].dtype)
            continue
        dz = _turn(s["d" + name].float().view(rows, -1, D), tab, case["R"], case["interleaved"], -1.0)
        dn = dz * w
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        out["d" + name] = dx.reshape(rows, -1).to(s[name].dtype)
        out["d" + name + "_weight"] = (dz * n).double().sum((0, 1)).to(s[name].dtype)
    return out


def _slots(s, case, seq, pos):
    page = s["block_table"].long()[seq, pos // case["page_rows"]]
    return page * case["page_rows"] + pos % case["page_rows"]


def _plain_append(s, case):
    rows, G, D, sr = s["k_new"].shape[0], case["G"], case["D"], case["scale_rows"]
    row = torch.arange(rows, device="cuda")
    q_start, kv = s["q_start"].long(), s["kv_len"].long()
    seq = torch.searchsorted(q_start, row, right=True) - 1
    pos = kv[seq] - q_start[seq + 1] + row
    slot = _slots(s, case, seq, pos)
    tab = s["table"][pos]

    def turned(x, weight):
        x = x.float().view(rows, -1, D)
        if weight is not None:
            x = _unit(x)[0] * weight.float()
        return _turn(x, tab, case["R"], case["interleaved"], 1.0)

    # Rows that the block of each sequence's first new position held before.
    ctx = kv - (q_start[1:] - q_start[:-1])
    old_pos = (ctx // sr * sr)[:, None] + torch.arange(sr, device="cuda")
    held = (old_pos < ctx[:, None]).nonzero()
    old_slot = _slots(s, case, held[:, 0], old_pos[held[:, 0], held[:, 1]])
    n_blocks = s["k_scales"].shape[0]
    kept = torch.zeros(n_blocks, dtype=torch.bool, device="cuda")
    kept[old_slot // sr] = True
    for name, x in (("k", turned(s["k_new"], s["k_weight"])), ("v", s["v_new"].float().view(rows, G, D))):
        codes, scales = s[name + "_pages"], s[name + "_scales"]
        amax = torch.zeros(n_blocks, G, device="cuda")
        amax.index_reduce_(0, slot // sr, x.abs().amax(-1), "amax")
        e_old = torch.where(kept[:, None], scales.int() - 127, -14)
        e = torch.maximum(e_old, _exponents(amax))
        old = codes[old_slot].view(torch.float8_e4m3fn).float().view(-1, G, D)
        old = old * torch.exp2((e_old - e)[old_slot // sr].float())[..., None]
        codes[old_slot] = old.view(-1, G * D).to(torch.float8_e4m3fn).view(torch.uint8)
        y = (x * torch.exp2(-e[slot // sr].float())[..., None]).clamp(-448.0, 448.0)
        codes[slot] = y.view(rows, -1).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[slot // sr] = (e + 127).to(torch.uint8)[slot // sr]
    out = _state8(s)
    if case["H"]:
        out["q"] = turned(s["q"], s["q_weight"]).view(rows, -1).to(s["q_out"].dtype)
    return out


def _values(s, case, name, slot):
    """What the cache's rows `slot` stand for, [rows, G, D] in 32 bits."""
    x = s[name + "_pages"][slot].view(torch.float8_e4m3fn).float().view(-1, case["G"], case["D"])
    return x * torch.exp2(s[name + "_scales"][slot // case["scale_rows"]].float() - 127.0)[..., None]


def _plain_read(s, case):
    row = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["starts"].long(), row, right=True) - 1
    slot = _slots(s, case, seq, s["first_pos"].long()[seq] + row - s["starts"].long()[seq])
    return {name: _values(s, case, name, slot).view(s["total"], -1).to(_DT[case["dtype"]]) for name in ("k", "v")}


def _plain_attend(s, case):
    H, G, D, pr = case["H"], case["G"], case["D"], case["page_rows"]
    out = torch.empty_like(s["q"])
    at = 0
    for i, (n, length) in enumerate(zip(s["new"], s["kv"])):
        pages = s["block_table"][i, :(length + pr - 1) // pr].long()
        slot = (pages[:, None] * pr + torch.arange(pr, device="cuda")).view(-1)[:length]
        if case["bits"] == 8:
            k, v = _values(s, case, "k", slot), _values(s, case, "v", slot)
        else:
            k, v = s["k_pages"][slot].float().view(-1, G, D), s["v_pages"][slot].float().view(-1, G, D)
        q = s["q"][at:at + n].float().view(n, G, H // G, D)
        sc = torch.matmul(q.permute(1, 2, 0, 3).reshape(G, -1, D), k.permute(1, 2, 0)) * (1.0 / math.sqrt(D))
        sc = sc.view(G, H // G, n, length)
        if case["softcap"]:
            sc = case["softcap"] * torch.tanh(sc / case["softcap"])
        p = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        if case["alibi"]:
            sc = sc - s["slopes"].view(G, H // G, 1, 1) * (p - j).abs().float()
        keep = j <= p
        if case["prefix"]:
            keep = keep | (j < s["prefix_len"][i])
        if case["window"]:
            keep = keep & ((j > p - case["window"]) | (j < case["sinks"]))
        sc = sc.masked_fill(~keep, float("-inf"))
        e = torch.exp(sc - sc.amax(-1, keepdim=True))
        w = e / e.sum(-1, keepdim=True)
        o = torch.matmul(w.view(G, -1, length), v.permute(1, 0, 2)).view(G, H // G, n, D)
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, H * D).to(out.dtype)
        at += n
    return out


_RUN_PLAIN = {"norm": _plain_norm, "append8": _plain_append, "read8": _plain_read, "attend": _plain_attend}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        return _norm64(s, case)
    if case["op"] == "append8":
        return _append64(s, case)
    if case["op"] == "read8":
        return _read64(s, case)
    if work(case)["flops"] > 8e12:
        return None
    return _attend64(s, case)


def _rotate64(x, pos, R, interleaved, inverse=False):
    """Each pair as a complex number times e^(i p theta), or its conjugate."""
    angle = pos.double()[:, None] * _theta(R)
    unit = torch.polar(torch.ones_like(angle), -angle if inverse else angle)[:, None, :]
    out = x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _norm64(s, case):
    rows, D, R, inter = case["rows"], case["D"], case["R"], case["interleaved"]
    out = {}
    for name in ("q", "k"):
        x, w = s[name].double().reshape(rows, -1, D), s[name + "_weight"].double()
        ms = x.pow(2).sum(-1, keepdim=True) / D + _EPS
        if not case["grad"]:
            out[name] = _rotate64(x * w / ms.sqrt(), s["pos"], R, inter).reshape(rows, -1)
            continue
        dz = _rotate64(s["d" + name].double().view(rows, -1, D), s["pos"], R, inter, True)
        dot = (dz * w * x).sum(-1, keepdim=True)
        out["d" + name] = (dz * w / ms.sqrt() - x * dot / (D * ms * ms.sqrt())).reshape(rows, -1)
        out["d" + name + "_weight"] = torch.einsum("rhd,rhd,rh->d", dz, x, ms[..., 0].rsqrt())
    return out


def _e4m3(x):
    """x rounded to the nearest e4m3 value, ties to the even one, saturated at 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _codes64(codes):
    """The values of e4m3 bytes, from their fields."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    size = torch.where(e > 0, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0), m * 2.0 ** -9)
    return torch.where(c >= 128, -size, size)


def _append64(s, case):
    G, D, pr, sr = case["G"], case["D"], case["page_rows"], case["scale_rows"]
    table = s["block_table"].tolist()
    slots, pos, groups = [], [], []  # groups: pool block, its rows held before, its new rows
    at = 0
    for i, (n, length) in enumerate(zip(s["new"], s["kv"])):
        ctx = length - n
        for first in range(ctx // sr * sr, length, sr):
            base = table[i][first // pr] * pr + first % pr
            held = max(0, ctx - first)
            end = min(sr, length - first)
            groups.append((base, held, at + first + held - ctx, end - held))
        for t in range(ctx, length):
            slots.append(table[i][t // pr] * pr + t % pr)
            pos.append(t)
        at += n
    slots, pos = torch.tensor(slots, device="cuda"), torch.tensor(pos, device="cuda")
    n = len(slots)

    def turned(x, w):
        x = x.double().view(n, -1, D)
        if w is not None:
            x = x * w.double() / (x.pow(2).mean(-1, keepdim=True) + _EPS).sqrt()
        return _rotate64(x, pos, case["R"], case["interleaved"])

    out = {}
    base, held, row0, count = (torch.tensor(v, device="cuda") for v in zip(*groups))
    of_row = torch.repeat_interleave(torch.arange(len(groups), device="cuda"), count)
    for name, x in (("k", turned(s["k_new"], s["k_weight"])), ("v", s["v_new"].double().view(n, G, D))):
        codes, scales = s[name + "_pages"].clone(), s[name + "_scales"]
        size = torch.zeros(len(groups), G, dtype=torch.float64, device="cuda")
        size.scatter_reduce_(0, of_row[:, None].expand(n, G), x.abs().amax(-1), "amax")
        e = torch.ceil(torch.log2((size / 448.0).clamp_min(2.0 ** -14))).clamp(-14, 7)
        before = scales[base // sr].double() - 127.0
        e = torch.where(held[:, None] > 0, torch.maximum(e, before), e)
        value = _codes64(codes).view(-1, G, D)
        grid = torch.arange(sr, device="cuda")
        which, offset = (grid[None, :] < held[:, None]).nonzero(as_tuple=True)
        old = base[which] + offset
        value[old] = _e4m3(value[old] * torch.exp2(before - e)[which][..., None])
        value[slots] = _e4m3((x / torch.exp2(e[of_row])[..., None]).clamp(-448.0, 448.0))
        out[name + "_pages"] = value.view(codes.shape)
        sizes = torch.exp2(scales.double() - 127.0)
        sizes[base // sr] = torch.exp2(e)
        out[name + "_scales"] = sizes
    if case["H"]:
        out["q"] = turned(s["q"], s["q_weight"]).view(n, -1)
    return out


def _rows64(s, case, name, slot, g=None):
    """Rows of the cache in 64 bits, of kv head g alone where it is given."""
    G, D = case["G"], case["D"]
    cols = slice(0, G * D) if g is None else slice(g * D, (g + 1) * D)
    if case.get("bits") == 16:
        return s[name + "_pages"][slot, cols].double()
    size = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"),
                       s[name + "_scales"][slot // case["scale_rows"]].int() - 127)
    size = size.repeat_interleave(D, 1)[:, cols]
    return _codes64(s[name + "_pages"][slot, cols]) * size


def _read64(s, case):
    out = {"k": [], "v": []}
    for i, (a, b) in enumerate(zip(s["first"], s["kv"])):
        t = torch.arange(a, b, device="cuda")
        slot = s["block_table"][i].long()[t // case["page_rows"]] * case["page_rows"] + t % case["page_rows"]
        for name in ("k", "v"):
            out[name].append(_rows64(s, case, name, slot))
    return {name: torch.cat(x) for name, x in out.items()}


def _attend64(s, case):
    """Query rows in blocks, one kv head at a time."""
    H, G, D, pr = case["H"], case["G"], case["D"], case["page_rows"]
    gs = H // G
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for i, (n, length) in enumerate(zip(s["new"], s["kv"])):
        t = torch.arange(length, device="cuda")
        slot = s["block_table"][i].long()[t // pr] * pr + t % pr
        for g in range(G):
            k_all, v_all = _rows64(s, case, "k", slot, g), _rows64(s, case, "v", slot, g)
            for b in range(0, n, 1024):
                m = min(1024, n - b)
                p = length - n + b + torch.arange(m, device="cuda").view(1, m, 1)
                end = length if case["prefix"] else length - n + b + m
                j = t[:end].view(1, 1, -1)
                ok = (j <= p) | (j < s["prefix"][i]) if case["prefix"] else j <= p
                if case["window"]:
                    ok = ok & ((p - j < case["window"]) | (j < case["sinks"]))
                q = s["q"][first + b:first + b + m, g * gs * D:(g + 1) * gs * D].double().view(m, gs, D).transpose(0, 1)
                x = q @ k_all[:end].t() / math.sqrt(D)
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if case["alibi"]:
                    h = torch.arange(g * gs, (g + 1) * gs, device="cuda", dtype=torch.float64)
                    slope = torch.exp2(-8.0 * (h + 1.0) / H).float().double()
                    x = x - slope.view(gs, 1, 1) * (p - j).abs()
                x = torch.where(ok, x, torch.full((), float("-inf"), dtype=torch.float64, device="cuda"))
                weight = torch.softmax(x, -1)
                out[first + b:first + b + m, g * gs * D:(g + 1) * gs * D] = \
                    (weight @ v_all[:end]).transpose(0, 1).reshape(m, gs * D)
        first += n
    return out
