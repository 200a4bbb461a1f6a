"""Allocating helpers over the C entry points (output tensors come from torch)."""
import math

import torch

from . import _binding as B


_SCALINGS = {"none": B.ATTN_ROPE_NONE, "linear": B.ATTN_ROPE_LINEAR, "ntk": B.ATTN_ROPE_NTK,
             "by_parts": B.ATTN_ROPE_BY_PARTS}


def rope_table(max_pos, head_dim, base=10000.0, device="cuda", stream=None, scaling=None, factor=1.0, orig_max_pos=0,
               beta_fast=32.0, beta_slow=1.0, attn_factor=1.0):
    """[max_pos, head_dim] RoPE table (cos of the head_dim/2 pair angles, then their sin).  For heads turned
    in part, head_dim is the turned part.  scaling ("none", "linear", "ntk", "by_parts") takes factor and,
    by parts, orig_max_pos, beta_fast, beta_slow; attn_factor multiplies every entry (see
    attn_rope_table_scaled in attn_gqa.h)."""
    t = torch.empty((max_pos, head_dim), device=device, dtype=torch.float32)
    with _on(t):
        if scaling is None:
            B.attn_rope_table(t, max_pos, head_dim, base, stream)
        else:
            if scaling not in _SCALINGS:
                raise ValueError("scaling must be one of %s" % ", ".join(sorted(_SCALINGS)))
            B.attn_rope_table_scaled(t, max_pos, head_dim, base, _SCALINGS[scaling], factor, orig_max_pos, beta_fast,
                                     beta_slow, attn_factor, stream)
    return t


def _on(x, *others):
    """The device of x as the current one for a call; every tensor of the call must be on it."""
    for o in others:
        if o is not None and o.device != x.device:
            raise ValueError("tensors of one call must be on one device, got %s and %s" % (x.device, o.device))
    return torch.cuda.device(x.device)


def _rows2d(x, name):
    """Row stride of a [rows, columns] tensor whose columns are contiguous."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("%s must be [rows, columns] with contiguous columns" % name)
    # The stride of a single row is never used, and torch may leave anything there.
    return max(x.stride(0), x.shape[1]) if x.shape[0] > 1 else x.shape[1]


def _rope(x, table, heads, positions, rot_dim, interleaved, out, inverse, stream):
    xs = _rows2d(x, "x")
    if heads < 1 or x.shape[1] % heads:
        raise ValueError("x has %d columns, not a multiple of %d heads" % (x.shape[1], heads))
    D = x.shape[1] // heads
    rot_dim = D if rot_dim is None else rot_dim
    if table.dim() != 2 or table.shape[1] != rot_dim or not table.is_contiguous():
        raise ValueError("table must be a contiguous [positions, %d] table of rope_table" % rot_dim)
    if positions is not None and positions.numel() != x.shape[0]:
        raise ValueError("positions must hold one position a row")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif out.shape != x.shape:
        raise ValueError("out must have the shape of x")
    with _on(x, table, positions, out):
        B.attn_rope_apply(x, out, x.shape[0], heads, D, rot_dim, xs, _rows2d(out, "out"),
                          B.ATTN_ROPE_INTERLEAVED if interleaved else B.ATTN_ROPE_HALF, positions, table, None, inverse,
                          stream)
    return out


def rope(x, table, heads, positions=None, rot_dim=None, interleaved=False, out=None, stream=None):
    """x [rows, heads*D] (fp32, bf16 or fp16; rows may be strided) turned by each row's position (row t
    at position t without `positions`).  rot_dim < D turns the first rot_dim columns of each head; out may be x."""
    return _rope(x, table, heads, positions, rot_dim, interleaved, out, False, stream)


def rope_backward(dy, table, heads, positions=None, rot_dim=None, interleaved=False, out=None, stream=None):
    """Gradient of rope's x for upstream dy."""
    return _rope(dy, table, heads, positions, rot_dim, interleaved, out, True, stream)


def forward(q, k, v, num_heads, num_kv_heads, mask=B.ATTN_CAUSAL, prec=B.ATTN_FP32, want_lse=True,
            stream=None, window=0, rope=None):
    """q [q_seq, H*D], k/v [kv_seq, G*D] (CUDA fp32) -> (out [q_seq, H*D], lse [q_seq, H, 2] or None).
    window > 0 keeps each row's last `window` keys; rope (a table from rope_table) turns q and k
    by their row positions first."""
    q_seq, kv_seq = q.shape[0], k.shape[0]
    D = q.shape[1] // num_heads
    out = torch.empty_like(q)
    lse = torch.empty((q_seq, num_heads, 2), device=q.device, dtype=torch.float32) if want_lse else None
    if rope is not None:
        B.attn_forward_rope(q, k, v, out, lse, q_seq, kv_seq, num_heads, num_kv_heads, D, mask, prec, window, rope,
                            None, stream)
    elif window:
        B.attn_forward_window(q, k, v, out, lse, q_seq, kv_seq, num_heads, num_kv_heads, D, mask, prec, window,
                              stream)
    else:
        B.attn_forward(q, k, v, out, lse, q_seq, kv_seq, num_heads, num_kv_heads, D, mask, prec, stream)
    return out, lse


def backward(q, k, v, out, lse, dout, num_heads, num_kv_heads, mask=B.ATTN_CAUSAL, window=0, stream=None):
    """Gradients (dq, dk, dv) of forward(q, k, v, ...)'s out for upstream dout, given its out and lse."""
    q_seq, kv_seq = q.shape[0], k.shape[0]
    D = q.shape[1] // num_heads
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    B.attn_backward(q, k, v, out, dout, lse, dq, dk, dv, q_seq, kv_seq, num_heads, num_kv_heads, D, mask,
                    B.ATTN_FP32, window, stream)
    return dq, dk, dv


def prefill(q_batch, k_cache, v_cache, n_queries, n_heads, n_kv_heads, head_dim, start_pos, q_base=0,
            scale=None, out=None, prec=B.ATTN_FP32, stream=None, window=0):
    """Causal prefill of rows q_base .. q_base+n_queries-1 of q_batch (row stride = its width)."""
    max_seq, kv_dim = k_cache.shape
    if out is None:
        out = torch.zeros((q_batch.shape[0], n_heads * head_dim), device=q_batch.device, dtype=torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    if window:
        B.attn_prefill_window(q_batch, k_cache, v_cache, out, n_queries, n_heads, n_kv_heads, head_dim, kv_dim,
                              max_seq, scale, start_pos, q_batch.shape[1], out.shape[1], q_base, prec, window, stream)
    else:
        B.attn_prefill(q_batch, k_cache, v_cache, out, n_queries, n_heads, n_kv_heads, head_dim, kv_dim, max_seq,
                       scale, start_pos, q_batch.shape[1], out.shape[1], q_base, prec, stream)
    return out


class DecodeState:
    """A decode workspace (zeroed once) and the device-resident kv_pos word."""

    def __init__(self, num_heads, num_kv_heads, head_dim, max_seq, device="cuda"):
        self.num_heads, self.num_kv_heads, self.head_dim, self.max_seq = num_heads, num_kv_heads, head_dim, max_seq
        nbytes = B.attn_decode_workspace_bytes(num_heads, num_kv_heads, head_dim, max_seq)
        if nbytes == 0:
            raise ValueError("unsupported decode sizes")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.kv_pos = torch.zeros(1, dtype=torch.int32, device=device)

    def set_pos(self, kv_pos):
        self.kv_pos.fill_(int(kv_pos))


def decode(state, q, k_cache, v_cache, out=None, stream=None, window=0):
    """One decode step at the position held in state.kv_pos (over its last
    `window` positions when window > 0)."""
    if out is None:
        out = torch.empty_like(q)
    if window:
        B.attn_decode_cached_window(q, k_cache, v_cache, state.kv_pos, out, state.num_heads, state.num_kv_heads,
                                    state.head_dim, state.max_seq, state.workspace, None, window, stream)
    else:
        B.attn_decode_cached(q, k_cache, v_cache, state.kv_pos, out, state.num_heads, state.num_kv_heads,
                             state.head_dim, state.max_seq, state.workspace, None, stream)
    return out


class PagedBatch:
    """A ragged batch over a paged cache: the device tensors that describe it and the attention's workspace.

    block_table [n_seqs, max_blocks], q_start [n_seqs + 1] and kv_len [n_seqs] are int32 CUDA tensors, kept
    and read on the device at each call (write into them between steps; see attn_gqa.h).  Calls
    that share a batch object must be ordered on one stream."""

    def __init__(self, block_table, q_start, kv_len, num_heads, num_kv_heads, head_dim, page_rows):
        if block_table.dim() != 2 or q_start.dim() != 1 or kv_len.dim() != 1 or \
                q_start.numel() != block_table.shape[0] + 1 or kv_len.numel() != block_table.shape[0]:
            raise ValueError("block_table [n, max_blocks], q_start [n + 1] and kv_len [n] do not fit together")
        self.block_table, self.q_start, self.kv_len = block_table, q_start, kv_len
        self.n_seqs, self.max_blocks = block_table.shape
        self.num_heads, self.num_kv_heads, self.head_dim, self.page_rows = num_heads, num_kv_heads, head_dim, page_rows
        with _on(block_table, q_start, kv_len):
            nbytes = B.attn_batch_paged_workspace_bytes(num_heads, num_kv_heads, head_dim)
        if nbytes == 0:
            raise ValueError("unsupported head sizes")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=block_table.device)

    def pool(self, k_pages, v_pages):
        """(kv_dim, num_pages) of two pools [num_pages * page_rows, kv_dim]."""
        if k_pages.shape != v_pages.shape or k_pages.dim() != 2 or k_pages.shape[0] % self.page_rows or \
                not k_pages.is_contiguous() or not v_pages.is_contiguous():
            raise ValueError("k_pages and v_pages must be contiguous [num_pages * page_rows, kv_dim] pools")
        return k_pages.shape[1], k_pages.shape[0] // self.page_rows


def append_paged(batch, k_new, v_new, k_pages, v_pages, q=None, q_out=None, table=None, rot_dim=None,
                 interleaved=False, stream=None):
    """Write the batch's new K (turned by `table`, when given) and V rows into the pages; with q, also
    return it turned, in the cache's type (q_out when given)."""
    kv_dim, num_pages = batch.pool(k_pages, v_pages)
    rows, D, G = k_new.shape[0], batch.head_dim, batch.num_kv_heads
    H = 0 if q is None else batch.num_heads
    for name, x, heads in (("k_new", k_new, G), ("v_new", v_new, G), ("q", q, H), ("q_out", q_out, H)):
        if x is not None and tuple(x.shape) != (rows, heads * D):
            raise ValueError("%s must be [%d, %d]" % (name, rows, heads * D))
    if q is not None and q_out is None:
        q_out = torch.empty((rows, H * D), dtype=k_pages.dtype, device=q.device)
    R = 0 if table is None else (D if rot_dim is None else rot_dim)
    if table is not None and (table.dim() != 2 or table.shape[1] != R or not table.is_contiguous()):
        raise ValueError("table must be a contiguous [positions, %d] table of rope_table" % R)
    with _on(k_pages, v_pages, k_new, v_new, q, q_out, table, batch.block_table):
        B.attn_append_paged(q, q_out, k_new, v_new, k_pages, v_pages, batch.block_table, batch.q_start, batch.kv_len,
                            rows, batch.n_seqs, H, G, D, kv_dim, _rows2d(q, "q") if H else 0,
                            _rows2d(q_out, "q_out") if H else 0, _rows2d(k_new, "k_new"), _rows2d(v_new, "v_new"),
                            batch.page_rows, num_pages, batch.max_blocks, R,
                            B.ATTN_ROPE_INTERLEAVED if interleaved else B.ATTN_ROPE_HALF, table, None, stream)
    return q_out


def attend_paged(batch, q, k_pages, v_pages, out=None, scale=None, window=0, softcap=0.0, alibi_slopes=None,
                 prefix_len=None, stream=None):
    """Attention of the batch's new tokens, q [rows, H*D] (bf16 or fp16), over its pages: the last `window`
    keys of each row (0 = all), scores capped by softcap * tanh(s / softcap) (0 = uncapped) and biased by
    -alibi_slopes[h] * distance, keys below prefix_len[s] visible to every row.  Rows of no sequence are
    left as they are in `out`."""
    kv_dim, num_pages = batch.pool(k_pages, v_pages)
    H, D = batch.num_heads, batch.head_dim
    if q.dim() != 2 or q.shape[1] != H * D:
        raise ValueError("q must be [rows, %d]" % (H * D))
    if out is None:
        out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    if alibi_slopes is not None and (alibi_slopes.numel() != H or not alibi_slopes.is_contiguous()):
        raise ValueError("alibi_slopes must hold one slope a head")
    if prefix_len is not None and prefix_len.numel() != batch.n_seqs:
        raise ValueError("prefix_len must hold one length a sequence")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on(k_pages, v_pages, q, out, alibi_slopes, prefix_len, batch.block_table):
        B.attn_batch_paged(q, k_pages, v_pages, out, batch.block_table, batch.q_start, batch.kv_len, q.shape[0],
                           batch.n_seqs, H, batch.num_kv_heads, D, kv_dim, _rows2d(q, "q"), _rows2d(out, "out"),
                           batch.page_rows, num_pages, batch.max_blocks, scale, window, softcap, alibi_slopes,
                           prefix_len, batch.workspace, None, stream)
    return out
