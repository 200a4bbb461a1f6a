"""Cases of the batched serving operators: rotary positions, appending to a
paged cache, and attention of each sequence's new tokens over its pages.

Each operator stands here in plain torch operations (32 bits, rounded once at
the end) and as the calls of this package that replace them; `own` picks which
of the two `run` makes.  `exact` gives the same results from the definitions
in 64 bits.

    rotary      pairs (i, i + R/2), or (2i, 2i + 1) when interleaved, of the
                first R columns of a head turn by the angle p theta_i at position p
    append      row i of sequence s belongs to position kv_len[s] - n_s + i, where
                n_s rows are new; K (and Q) are turned, K and V go to their page
    attention   the row at position p attends keys
                [max(0, p + 1 - window), max(p + 1, min(prefix, kv_len))) with
                score cap * tanh(scale q.k / cap) - slope_h |p - j|
"""
import math
import random

import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_ESIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


# ------------------------------------------------------------------ cases
def listed():
    """Twelve cases.  32 query heads over 8 kv heads of 128 columns are the
    repository's benchmark heads; 16384 its decode cache, 8192 its forward."""
    return [
        # A packed QKV projection of a training or prefill step, its Q and K heads turned.
        _rope("rope_packed_bf16", rows=8192, heads=40, D=128, R=128, stride=6144),
        # The gradient of a model that turns part of each head, interleaved, scaled for long contexts.
        _rope("rope_grad_fp32_part", rows=4099, heads=12, D=80, R=32, stride=960, dtype="fp32", interleaved=True,
              grad=True, scaling="by_parts", pos_max=16384),
        # One token of each of a few sequences: latency.
        _rope("rope_step_fp16", rows=5, heads=10, D=64, R=64, stride=640, dtype="fp16", pos_max=16384),
        # A serving step: one token of 64 sequences, Q turned in the same call.
        _append("append_step_bf16", n_seqs=64, new=(1, 1), ctx=(1, 2047), page_rows=16),
        # Chunks of prompts from an fp32 model into a bf16 cache.
        _append("append_chunks_fp32_to_bf16", n_seqs=4, new=(2048, 2048), ctx=(0, 511), page_rows=64, src="fp32"),
        # Ragged chunks with odd heads, an odd page and part of the head turned; no Q.
        _append("append_odd_fp16", n_seqs=7, new=(1, 301), ctx=(0, 999), page_rows=24, dtype="fp16", src="fp16", H=0,
                G=3, D=96, R=48, interleaved=True),
        # One sequence, one token, a short cache: the latency of a chat turn.
        _attend("decode_one_bf16", n_seqs=1, new=(1, 1), ctx=(1535, 1535), page_rows=64),
        # A serving step of 64 sequences of very different lengths in small pages.
        _attend("decode_batch_bf16", n_seqs=64, new=(1, 1), ctx=(0, 16383), page_rows=16),
        # Capped scores and a sliding window, seven query heads a kv head.
        _attend("decode_cap_window_fp16", n_seqs=33, new=(1, 1), ctx=(100, 16000), page_rows=32, dtype="fp16", H=14,
                G=2, D=64, softcap=30.0, window=4096),
        # A chunk of a prompt behind a long cache: few rows, many keys.
        _attend("chunk_long_bf16", n_seqs=2, new=(512, 512), ctx=(16384, 32000), page_rows=64),
        # A whole prompt.
        _attend("prefill_bf16", n_seqs=1, new=(8192, 8192), ctx=(0, 0), page_rows=64),
        # Chunks and single tokens mixed, distance bias, a prefix that every row sees.
        _attend("mixed_bias_prefix_fp16", n_seqs=17, new=(1, 777), ctx=(0, 4097), page_rows=128, dtype="fp16", H=16,
                G=16, D=128, alibi=True, prefix=True),
    ]


def _rope(name, rows, heads, D, R, stride, dtype="bf16", interleaved=False, grad=False, scaling="none", pos_max=None):
    c = dict(op="rope", rows=rows, heads=heads, D=D, R=R, stride=stride, dtype=dtype, interleaved=interleaved,
             grad=grad, scaling=scaling, pos_max=pos_max or rows)
    return dict(c, name=name) if name else c


def _append(name, n_seqs, new, ctx, page_rows, dtype="bf16", src="bf16", H=32, G=8, D=128, R=None, interleaved=False,
            ragged=1):
    c = dict(op="append", n_seqs=n_seqs, new_min=new[0], new_max=new[1], ctx_min=ctx[0], ctx_max=ctx[1],
             page_rows=page_rows, dtype=dtype, src=src, H=H, G=G, D=D, R=D if R is None else R,
             interleaved=interleaved, ragged=ragged)
    return dict(c, name=name) if name else c


def _attend(name, n_seqs, new, ctx, page_rows, dtype="bf16", H=32, G=8, D=128, softcap=0.0, window=0, alibi=False,
            prefix=False, ragged=2):
    c = dict(op="attend", n_seqs=n_seqs, new_min=new[0], new_max=new[1], ctx_min=ctx[0], ctx_max=ctx[1],
             page_rows=page_rows, dtype=dtype, H=H, G=G, D=D, softcap=softcap, window=window, alibi=alibi,
             prefix=prefix, ragged=ragged)
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "append", "attend", "attend"])
        ragged = rng.randrange(1 << 30)
        if op == "rope":
            D = rng.choice([64, 128, 80, 96, 50, rng.randrange(8, 129, 2)])
            R = rng.choice([D, D // 4 * 2, rng.randrange(2, D + 1, 2)])
            heads = _log(rng, 1, 48)
            rows = _log(rng, 1, 16384)
            c = _rope(None, rows, heads, D, max(R, 2), heads * D + rng.choice([0, 8, 1, D]),
                      rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5, rng.random() < 0.4,
                      rng.choice(["none", "linear", "ntk", "by_parts"]), max(rows, _log(rng, 64, 131072)))
            if c["R"] <= 2 and c["scaling"] == "ntk":
                continue  # the rescaled base needs more than one pair
            limit = work(listed()[0])["bytes"]
        elif op == "append":
            D = rng.choice([64, 128, 96, 80])
            G = rng.choice([1, 2, 3, 4, 8])
            src, dtype = rng.choice([("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"), ("fp32", "fp32"),
                                     ("fp32", "fp16")])
            hi = rng.choice([1, _log(rng, 1, 2048)])
            c = _append(None, _log(rng, 1, 128), (1, hi), (0, _log(rng, 1, 2048)),
                        rng.choice([16, 32, 64, 128, rng.randrange(1, 100)]), dtype, src,
                        G * rng.choice([0, 1, 2, 4, 5, 8]), G, D, rng.choice([D, D // 2, D // 4]),
                        rng.random() < 0.4, ragged)
            limit = work(listed()[4])["bytes"]
        else:
            D = rng.choice([64, 128, 128, 64, 96, 80])
            G = rng.choice([1, 2, 4, 8])
            hi = rng.choice([1, 1, _log(rng, 1, 2048)])
            c = _attend(None, _log(rng, 1, 96), (1, hi), (0, _log(rng, 1, 32768)),
                        rng.choice([16, 32, 64, 128, 256, rng.randrange(1, 100)]), rng.choice(["bf16", "fp16"]),
                        G * rng.choice([1, 2, 4, 8, 3, 7, 16]), G, D, rng.choice([0.0, 0.0, 30.0, 50.0]),
                        rng.choice([0, 0, _log(rng, 1, 8192)]), rng.random() < 0.3, rng.random() < 0.25, ragged)
            w, big = work(c), work(listed()[10])
            if w["flops"] > big["flops"] or w["bytes"] > work(listed()[7])["bytes"]:
                continue
            return c
        if work(c)["bytes"] <= limit:
            return c


def _lengths(case):
    """New rows, total length and prefix of each sequence, spread over their ranges."""
    rng = random.Random(case["ragged"])
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["n_seqs"])]
    kv = [n + rng.randint(case["ctx_min"], case["ctx_max"]) for n in new]
    prefix = [rng.randint(0, n) for n in kv]
    return new, kv, prefix


def _window_of(case, p, kv, prefix):
    """Keys [lo, hi) of the row at position p of a sequence of kv positions."""
    hi = max(p + 1, min(prefix, kv)) if case["prefix"] else p + 1
    lo = max(0, p + 1 - case["window"]) if case["window"] else 0
    return lo, hi


def work(case):
    if case["op"] == "rope":
        x = case["rows"] * case["heads"] * case["D"] * _ESIZE[case["dtype"]]
        table = min(case["rows"], case["pos_max"]) * case["R"] * 4
        return {"bytes": 2 * x + table + 4 * case["rows"], "flops": 3 * case["rows"] * case["heads"] * case["R"]}
    new, kv, prefix = _lengths(case)
    rows = sum(new)
    D, H, G = case["D"], case["H"], case["G"]
    if case["op"] == "append":
        io = _ESIZE[case["src"]] + _ESIZE[case["dtype"]]
        return {"bytes": rows * ((2 * G + H) * D * io + case["R"] * 4),
                "flops": 3 * rows * (G + H) * case["R"]}
    pairs = keys = 0
    for n, length, pre in zip(new, kv, prefix):
        first, hi_all = length, 0
        for p in range(length - n, length):
            lo, hi = _window_of(case, p, length, pre)
            pairs += hi - lo
            first, hi_all = min(first, lo), max(hi_all, hi)
        keys += hi_all - first
    es = _ESIZE[case["dtype"]]
    return {"bytes": (2 * keys * G + 2 * rows * H) * D * es, "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ inputs
_BASE = 10000.0
_SCALE = dict(factor=4.0, orig_max_pos=4096, beta_fast=32.0, beta_slow=1.0)


def _theta(R, scaling):
    """Angle per position of each of the R/2 pairs, 64 bits."""
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    f = _SCALE["factor"]
    if scaling == "ntk":
        return (_BASE * f ** (R / (R - 2.0))) ** (-2.0 * i / R)
    th = _BASE ** (-2.0 * i / R)
    if scaling == "linear":
        return th / f
    if scaling == "by_parts":
        turns = _SCALE["orig_max_pos"] * th / (2.0 * math.pi)
        keep = ((turns - _SCALE["beta_slow"]) / (_SCALE["beta_fast"] - _SCALE["beta_slow"])).clamp(0.0, 1.0)
        return th * (keep + (1.0 - keep) / f)
    return th


def _attn_factor(scaling):
    """The temperature that scaled tables carry on cos and sin."""
    return 0.1 * math.log(_SCALE["factor"]) + 1.0 if scaling == "by_parts" else 1.0


def _table(max_pos, R, scaling):
    """[max_pos, R]: cos of the R/2 pair angles of each position, then their sin."""
    if own:
        import attention_gqa_online_gb300 as A
        if scaling == "none":
            return A.rope_table(max_pos, R, _BASE)
        return A.rope_table(max_pos, R, _BASE, scaling=scaling, attn_factor=_attn_factor(scaling), **_SCALE)
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * _theta(R, scaling)
    return (torch.cat([ang.cos(), ang.sin()], 1) * _attn_factor(scaling)).float()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        return out.normal_(generator=g)

    s = {"case": case}
    if case["op"] == "rope":
        dt = _DT[case["dtype"]]
        base = randn(case["rows"], case["stride"], dtype=dt)
        s["x"] = base[:, :case["heads"] * case["D"]]
        pos = torch.randint(0, case["pos_max"], (case["rows"],), generator=g, device="cuda")
        if case["pos_max"] == case["rows"]:
            pos = torch.arange(case["rows"], device="cuda")  # a prompt from its first token
        s["pos"] = pos.to(torch.int32)
        return s
    new, kv, prefix = _lengths(case)
    pr, kv_dim = case["page_rows"], case["G"] * case["D"]
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
    dt = _DT[case["dtype"]]
    s["k_pages"] = randn(num_pages * pr, kv_dim, dtype=dt)
    s["v_pages"] = randn(num_pages * pr, kv_dim, dtype=dt)
    s["block_table"] = table.cuda()
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["new"], s["kv"], s["prefix"], s["num_pages"] = new, kv, prefix, num_pages
    rows = starts[-1]
    if case["op"] == "append":
        src = _DT[case["src"]]
        s["k_new"] = randn(rows, kv_dim, dtype=src)
        s["v_new"] = randn(rows, kv_dim, dtype=src)
        s["q"] = randn(rows, case["H"] * case["D"], dtype=src) if case["H"] else None
    else:
        s["q"] = randn(rows, case["H"] * case["D"], dtype=dt)
        if case["alibi"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["H"] + 1, device="cuda", dtype=torch.float32) / case["H"])
        if case["prefix"]:
            s["prefix_len"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        s["table"] = _table(case["pos_max"], case["R"], case["scaling"])
        s["out"] = torch.empty(case["rows"], case["heads"] * case["D"], dtype=s["x"].dtype, device="cuda")
        return s
    if case["op"] == "append":
        s["table"] = _table(max(s["kv"]), case["R"], "none")
        if case["H"]:
            s["q_out"] = torch.empty(s["q"].shape, dtype=_DT[case["dtype"]], device="cuda")
    else:
        s["out"] = torch.empty_like(s["q"])
    if own:
        import attention_gqa_online_gb300 as A
        s["batch"] = A.PagedBatch(s["block_table"], s["q_start"], s["kv_len"], max(case["H"], case["G"]), case["G"],
                                  case["D"], case["page_rows"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _RUN_OWN[case["op"]](state, case)
    return _RUN_PLAIN[case["op"]](state, case)


def _own_rope(s, case):
    import attention_gqa_online_gb300 as A
    call = A.rope_backward if case["grad"] else A.rope
    return call(s["x"], s["table"], case["heads"], positions=s["pos"], rot_dim=case["R"],
                interleaved=case["interleaved"], out=s["out"])


def _own_append(s, case):
    import attention_gqa_online_gb300 as A
    A.append_paged(s["batch"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], q=s["q"], q_out=s.get("q_out"),
                   table=s["table"], rot_dim=case["R"], interleaved=case["interleaved"])
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if case["H"]:
        out["q"] = s["q_out"]
    return out


def _own_attend(s, case):
    import attention_gqa_online_gb300 as A
    return A.attend_paged(s["batch"], s["q"], s["k_pages"], s["v_pages"], out=s["out"], window=case["window"],
                          softcap=case["softcap"], alibi_slopes=s.get("slopes"), prefix_len=s.get("prefix_len"))


_RUN_OWN = {"rope": _own_rope, "append": _own_append, "attend": _own_attend}


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


def _plain_rope(s, case):
    x = s["x"].float().view(case["rows"], case["heads"], case["D"]) if s["x"].is_contiguous() else \
        s["x"].float().reshape(case["rows"], case["heads"], case["D"])
    y = _turn(x, s["table"][s["pos"].long()], case["R"], case["interleaved"], -1.0 if case["grad"] else 1.0)
    return y.reshape(case["rows"], -1).to(s["x"].dtype)


def _plain_append(s, case):
    rows, D = s["k_new"].shape[0], case["D"]
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(s["q_start"].long(), row, right=True) - 1
    pos = s["kv_len"].long()[seq] - s["q_start"].long()[seq + 1] + row
    page = s["block_table"].long()[seq, pos // case["page_rows"]]
    slot = page * case["page_rows"] + pos % case["page_rows"]
    tab = s["table"][pos]
    k = _turn(s["k_new"].float().view(rows, -1, D), tab, case["R"], case["interleaved"], 1.0)
    s["k_pages"][slot] = k.view(rows, -1).to(s["k_pages"].dtype)
    s["v_pages"][slot] = s["v_new"].float().to(s["v_pages"].dtype)
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if case["H"]:
        q = _turn(s["q"].float().view(rows, -1, D), tab, case["R"], case["interleaved"], 1.0)
        out["q"] = q.view(rows, -1).to(s["k_pages"].dtype)
    return out


def _plain_attend(s, case):
    H, G, D, pr = case["H"], case["G"], case["D"], case["page_rows"]
    out = torch.empty_like(s["q"])
    at = 0
    for i, (n, length) in enumerate(zip(s["new"], s["kv"])):
        pages = s["block_table"][i, :(length + pr - 1) // pr].long()
        k = s["k_pages"].view(-1, pr, G * D)[pages].view(-1, G, D)[:length].float()
        v = s["v_pages"].view(-1, pr, G * D)[pages].view(-1, G, D)[:length].float()
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
            keep = keep & (j > p - case["window"])
        sc = sc.masked_fill(~keep, float("-inf"))
        e = torch.exp(sc - sc.amax(-1, keepdim=True))
        w = e / e.sum(-1, keepdim=True)
        o = torch.matmul(w.view(G, -1, length), v.permute(1, 0, 2)).view(G, H // G, n, D)
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, H * D).to(out.dtype)
        at += n
    return out


_RUN_PLAIN = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        z = _rotate64(s["x"].double().reshape(case["rows"], case["heads"], case["D"]), s["pos"], case["R"],
                      case["interleaved"], case["scaling"], case["grad"])
        return z.reshape(case["rows"], -1)
    if case["op"] == "append":
        return _append64(s, case)
    if work(case)["flops"] > 8e12:
        return None
    return _attend64(s, case)


def _rotate64(x, pos, R, interleaved, scaling, inverse):
    """Each pair as a complex number times m e^(i p theta), or its conjugate."""
    angle = pos.double()[:, None] * _theta(R, scaling)
    unit = torch.polar(torch.full_like(angle, _attn_factor(scaling)), -angle if inverse else angle)[:, None, :]
    out = x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _append64(s, case):
    pr, D = case["page_rows"], case["D"]
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    table = s["block_table"].tolist()
    slots, pos = [], []
    for i, (n, length) in enumerate(zip(s["new"], s["kv"])):
        for t in range(length - n, length):
            slots.append(table[i][t // pr] * pr + t % pr)
            pos.append(t)
    slots, pos = torch.tensor(slots, device="cuda"), torch.tensor(pos, device="cuda")
    n = len(slots)

    def turned(x):
        return _rotate64(x.double().view(n, -1, D), pos, case["R"], case["interleaved"], "none", False).view(n, -1)

    k_pages[slots] = turned(s["k_new"])
    v_pages[slots] = s["v_new"].double()
    out = {"k_pages": k_pages, "v_pages": v_pages}
    if case["H"]:
        out["q"] = turned(s["q"])
    return out


def _attend64(s, case):
    """Query rows in blocks, one kv head at a time, each block over the keys it can see."""
    H, G, D, pr = case["H"], case["G"], case["D"], case["page_rows"]
    gs = H // G
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for i, (n, length) in enumerate(zip(s["new"], s["kv"])):
        t = torch.arange(length, device="cuda")
        slot = s["block_table"][i].long()[t // pr] * pr + t % pr
        for b in range(0, n, 1024):
            m = min(1024, n - b)
            p = length - n + b + torch.arange(m, device="cuda").view(1, m, 1)
            end = length if case["prefix"] else length - n + b + m
            begin = max(0, length - n + b + 1 - case["window"]) if case["window"] else 0
            j = t[begin:end].view(1, 1, -1)
            ok = (j <= p) | (j < s["prefix"][i]) if case["prefix"] else j <= p
            if case["window"]:
                ok = ok & (p - j < case["window"])
            for g in range(G):
                k = s["k_pages"][slot[begin:end], g * D:(g + 1) * D].double()
                v = s["v_pages"][slot[begin:end], g * D:(g + 1) * D].double()
                q = s["q"][first + b:first + b + m, g * gs * D:(g + 1) * gs * D].double().view(m, gs, D).transpose(0, 1)
                x = q @ k.t() / math.sqrt(D)
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if case["alibi"]:
                    h = torch.arange(g * gs, (g + 1) * gs, device="cuda", dtype=torch.float64)
                    slope = torch.exp2(-8.0 * (h + 1.0) / H).float().double()
                    x = x - slope.view(gs, 1, 1) * (p - j).abs()
                x = torch.where(ok, x, torch.full((), float("-inf"), dtype=torch.float64, device="cuda"))
                weight = torch.softmax(x, -1)
                out[first + b:first + b + m, g * gs * D:(g + 1) * gs * D] = \
                    (weight @ v).transpose(0, 1).reshape(m, gs * D)
        first += n
    return out
