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
    if scaling is None and (factor != 1.0 or orig_max_pos != 0 or beta_fast != 32.0 or beta_slow != 1.0):
        raise ValueError("factor, orig_max_pos, beta_fast and beta_slow need a scaling")
    if scaling is None and attn_factor != 1.0:
        scaling = "none"
    _count32("orig_max_pos", orig_max_pos)
    if scaling is not None and scaling not in _SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(sorted(_SCALINGS)))
    t = _new(torch.empty, (max_pos, head_dim), torch.float32, device, stream)
    with _on(t):
        if scaling is None:
            B.attn_rope_table(t, max_pos, head_dim, base, stream)
        else:
            B.attn_rope_table_scaled(t, max_pos, head_dim, base, _SCALINGS[scaling], factor, orig_max_pos, beta_fast,
                                     beta_slow, attn_factor, stream)
    return t


def _on(x, *others):
    """The device of x as the current one for a call; every tensor of the call must be on it."""
    _same_device(x.get_device(), *others)
    return torch.cuda.device(x.device)


# The calls below are made once a layer of a serving step, where a microsecond of Python counts as much as one on
# the GPU: they check with the cheapest queries and hand addresses to the library directly.
_CODES = {torch.float32: B.ATTN_DT_F32, torch.bfloat16: B.ATTN_DT_BF16, torch.float16: B.ATTN_DT_F16}
_INT32 = (torch.int32, torch.uint32)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _same_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors of one call must be on one CUDA device, got cuda:%d and %s" % (index, t.device)
                             if index >= 0 else "tensors must be in device memory, got %s" % t.device)


def _count32(name, value):
    """Checks what ctypes would cut to 32 bits."""
    if not 0 <= value < 1 << 32:
        raise ValueError("%s must be from 0 to 2^32 - 1, got %d" % (name, value))


def _code(x, name):
    code = _CODES.get(x.dtype)
    if code is None:
        raise ValueError("%s must be float32, bfloat16 or float16, got %s" % (name, x.dtype))
    return code


def _like(dtype, name, x):
    if x is not None and x.dtype != dtype:
        raise ValueError("%s has type %s, unlike the tensors it goes with (%s)" % (name, x.dtype, dtype))


def _int32(x, name):
    """Address of a contiguous tensor of 32-bit integers, or None."""
    if x is None:
        return None
    if x.dtype not in _INT32 or not x.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of 32-bit integers" % name)
    return x.data_ptr()


def _handle(stream, index):
    """Raw stream of a call on device `index`."""
    if index < 0:
        raise ValueError("tensors must be in device memory")
    if stream is None:
        return _raw_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _run(where, fn, index, stream, args):
    """Calls library function `fn` with `args` and the raw stream, on device `index`."""
    if _current_device() == index:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            code = fn(*args, stream)
    if code:
        raise B.AttnError(code, where)


def _new(make, shape, dtype, device, stream):
    """A result made by torch on the call's stream: the memory and a fill belong to that stream's order."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream, device) if isinstance(stream, int) else stream):
        return make(shape, dtype=dtype, device=device)


def _stream_object(raw, device):
    return torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)


def _rows2d(x, name):
    """(rows, columns, row stride) of a [rows, columns] tensor whose columns are contiguous."""
    shape = x.shape
    if len(shape) == 2:
        rows, columns = shape
        stride, one = x.stride()
        if one == 1 or columns < 2:
            if rows < 2:  # the stride of a single row is never used, and torch may leave anything there
                stride = columns
            if rows >> 32 or stride >> 32:
                raise ValueError("%s has more rows, or rows farther apart, than 32 bits count" % name)
            return rows, columns, stride
    raise ValueError("%s must be [rows, columns] with contiguous columns" % name)


def _table(table, rot_dim):
    """(address, rows) of a rotary table, or (None, 0)."""
    if table is None:
        return None, 0
    shape = table.shape
    if len(shape) != 2 or shape[1] != rot_dim or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table must be a contiguous float32 [positions, %d] table of rope_table" % rot_dim)
    return table.data_ptr(), shape[0]


def _rope(x, table, heads, positions, rot_dim, interleaved, out, inverse, stream):
    rows, columns, xs = _rows2d(x, "x")
    if heads < 1 or columns % heads:
        raise ValueError("x has %d columns, not a multiple of %d heads" % (columns, heads))
    D = columns // heads
    if rot_dim is None:
        rot_dim = D
    code = _code(x, "x")
    tab, tab_rows = _table(table, rot_dim)
    pos = _int32(positions, "positions")
    if pos is not None and positions.numel() != rows:
        raise ValueError("positions must hold one position a row")
    index = x.get_device()
    if out is None:
        out = _new(torch.empty, (rows, columns), x.dtype, x.device, stream)
        ys = columns
    else:
        out_rows, out_columns, ys = _rows2d(out, "out")
        if out_rows != rows or out_columns != columns:
            raise ValueError("out must have the shape of x")
        _like(x.dtype, "out", out)
        _same_device(index, out)
    _same_device(index, table, positions)
    _run("attn_rope_apply", B.load_library().attn_rope_apply, index, _handle(stream, index),
         (x.data_ptr(), out.data_ptr(), code, rows, heads, D, rot_dim, xs, ys, 1 if interleaved else 0, pos, tab,
          tab_rows, 1 if inverse else 0))
    return out


def rope(x, table, heads, positions=None, rot_dim=None, interleaved=False, out=None, stream=None):
    """x [rows, heads*D] (fp32, bf16 or fp16; rows may be strided) turned by each row's position (row t
    at position t without `positions`).  rot_dim < D turns the first rot_dim columns of each head; out may be x."""
    return _rope(x, table, heads, positions, rot_dim, interleaved, out, False, stream)


def rope_backward(dy, table, heads, positions=None, rot_dim=None, interleaved=False, out=None, stream=None):
    """Gradient of rope's x for upstream dy."""
    return _rope(dy, table, heads, positions, rot_dim, interleaved, out, True, stream)


def _rows_out(out, like, shape, name, stream, make=torch.empty):
    """(tensor, row stride) of a result like `like`, allocated when out is None."""
    if out is None:
        return _new(make, shape, like.dtype, like.device, stream), shape[1]
    rows, columns, stride = _rows2d(out, name)
    if (rows, columns) != shape:
        raise ValueError("%s must be [%d, %d]" % ((name,) + shape))
    _like(like.dtype, name, out)
    return out, stride


def _heads2d(x, heads, name):
    rows, columns, stride = _rows2d(x, name)
    if heads < 1 or columns % heads:
        raise ValueError("%s has %d columns, not a multiple of %d heads" % (name, columns, heads))
    return rows, columns // heads, stride


def _weights(D, q_weight, k_weight):
    """(type code, addresses) of two weight vectors, either of them None (code 0 without any)."""
    code, ptr = None, [None, None]
    for i, w in enumerate((q_weight, k_weight)):
        if w is None:
            continue
        name = "k_weight" if i else "q_weight"
        if w.shape != (D,) or not w.is_contiguous():
            raise ValueError("%s must be a contiguous vector of %d" % (name, D))
        if code is None:
            code = _code(w, name)
        elif _CODES.get(w.dtype) != code:
            raise ValueError("q_weight and k_weight must have one type")
        ptr[i] = w.data_ptr()
    return code or 0, ptr[0], ptr[1]


def _ptr(x):
    return None if x is None else x.data_ptr()


def _norm_sizes(q, k, num_heads, num_kv_heads, q_weight, k_weight, table, positions, rot_dim):
    rows, D, qs = _heads2d(q, num_heads, "q")
    k_rows, k_D, ks = _heads2d(k, num_kv_heads, "k")
    if k_rows != rows or k_D != D:
        raise ValueError("q and k must have the same rows and the same head dimension")
    _like(q.dtype, "k", k)
    w_code, wq, wk = _weights(D, q_weight, k_weight)
    if table is None:
        if rot_dim:
            raise ValueError("a turn needs a table")
        rot_dim = 0
    elif rot_dim is None:
        rot_dim = D
    tab, tab_rows = _table(table, rot_dim)
    pos = _int32(positions, "positions")
    if pos is not None and positions.numel() != rows:
        raise ValueError("positions must hold one position a row")
    return rows, D, qs, ks, w_code, wq, wk, rot_dim, tab, tab_rows, pos


def qk_norm_rope(q, k, num_heads, num_kv_heads, q_weight=None, k_weight=None, table=None, positions=None, rot_dim=None,
                 interleaved=False, eps=1e-6, q_out=None, k_out=None, stream=None):
    """q [rows, H*D] and k [rows, G*D] (fp32, bf16 or fp16; rows may be strided) with each head normed by its
    root mean square, multiplied by its weight vector [D] (None: ones) and turned by its row's position (row t
    at t without `positions`; no table: not turned).  Returns (q_out, k_out), which may be the inputs."""
    rows, D, qs, ks, w_code, wq, wk, rot_dim, tab, tab_rows, pos = _norm_sizes(
        q, k, num_heads, num_kv_heads, q_weight, k_weight, table, positions, rot_dim)
    code, index = _code(q, "q"), q.get_device()
    q_out, qos = _rows_out(q_out, q, (rows, num_heads * D), "q_out", stream)
    k_out, kos = _rows_out(k_out, k, (rows, num_kv_heads * D), "k_out", stream)
    _same_device(index, k, q_out, k_out, q_weight, k_weight, table, positions)
    _run("attn_qk_norm_rope", B.load_library().attn_qk_norm_rope, index, _handle(stream, index),
         (q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), wq, wk, code, w_code,
          rows, num_heads, num_kv_heads, D, qs, ks, qos, kos, eps, rot_dim, 1 if interleaved else 0, pos, tab,
          tab_rows))
    return q_out, k_out


_norm_workspace = {}  # bytes by (device, head dimension)


def qk_norm_rope_backward(dq, dk, q, k, num_heads, num_kv_heads, q_weight=None, k_weight=None, table=None,
                          positions=None, rot_dim=None, interleaved=False, eps=1e-6, dq_out=None, dk_out=None,
                          stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of qk_norm_rope's q, k and weights (None for a weight that is None)
    for upstream dq, dk of its results.  dq_out and dk_out take the first two; they may be dq and dk, or q and k."""
    rows, D, qs, ks, w_code, wq, wk, rot_dim, tab, tab_rows, pos = _norm_sizes(
        q, k, num_heads, num_kv_heads, q_weight, k_weight, table, positions, rot_dim)
    code, index = _code(q, "q"), q.get_device()
    strides = []
    for name, x, heads in (("dq", dq, num_heads), ("dk", dk, num_kv_heads)):
        x_rows, x_D, stride = _heads2d(x, heads, name)
        if x_rows != rows or x_D != D:
            raise ValueError("%s must have the shape of %s" % (name, name[1]))
        _like(q.dtype, name, x)
        strides.append(stride)
    dq_out, dqos = _rows_out(dq_out, q, (rows, num_heads * D), "dq_out", stream)
    dk_out, dkos = _rows_out(dk_out, k, (rows, num_kv_heads * D), "dk_out", stream)
    _same_device(index, dq, dk, k, dq_out, dk_out, q_weight, k_weight, table, positions)
    raw = _handle(stream, index)
    dw = [None if w is None else _new(torch.empty, (D,), w.dtype, w.device, stream) for w in (q_weight, k_weight)]
    workspace, nbytes = None, 0
    if dw[0] is not None or dw[1] is not None:
        nbytes = _norm_workspace.get((index, D))
        if nbytes is None:
            with torch.cuda.device(index):
                nbytes = _norm_workspace[index, D] = B.attn_qk_norm_rope_backward_workspace_bytes(D)
        workspace = _new(torch.empty, (nbytes,), torch.uint8, q.device, stream)
    _run("attn_qk_norm_rope_backward", B.load_library().attn_qk_norm_rope_backward, index, raw,
         (dq.data_ptr(), dk.data_ptr(), q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(),
          wq, wk, _ptr(dw[0]), _ptr(dw[1]), code, w_code, rows, num_heads, num_kv_heads, D,
          strides[0], strides[1], qs, ks, dqos, dkos, eps, rot_dim, 1 if interleaved else 0, pos, tab, tab_rows,
          _ptr(workspace), nbytes))
    return dq_out, dk_out, dw[0], dw[1]


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
    that share a batch object, or a workspace (which may be set to another batch's), must be ordered on one
    stream, which need not be the one that the object was made on."""

    def __init__(self, block_table, q_start, kv_len, num_heads, num_kv_heads, head_dim, page_rows):
        if block_table.dim() != 2 or q_start.dim() != 1 or kv_len.dim() != 1 or \
                q_start.numel() != block_table.shape[0] + 1 or kv_len.numel() != block_table.shape[0]:
            raise ValueError("block_table [n, max_blocks], q_start [n + 1] and kv_len [n] do not fit together")
        self._index = block_table.get_device()
        if self._index < 0:
            raise ValueError("block_table, q_start and kv_len must be in device memory")
        self.n_seqs, self.max_blocks = block_table.shape
        self.block_table, self.q_start, self.kv_len = block_table, q_start, kv_len
        self.num_heads, self.num_kv_heads, self.head_dim, self.page_rows = num_heads, num_kv_heads, head_dim, page_rows
        with _on(block_table, q_start, kv_len):
            nbytes = B.attn_batch_paged_workspace_bytes(num_heads, num_kv_heads, head_dim)
        if nbytes == 0:
            raise ValueError("unsupported head sizes")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=block_table.device)

    def __setattr__(self, name, value):
        # The tensors are checked when they are set, so that a step need not check them again.
        if name in ("block_table", "q_start", "kv_len"):
            _int32(value, name)
            _same_device(self._index, value)
            shape = {"block_table": (self.n_seqs, self.max_blocks), "q_start": (self.n_seqs + 1,),
                     "kv_len": (self.n_seqs,)}[name]
            if value.shape != shape:
                raise ValueError("%s must be %s, got %s" % (name, list(shape), list(value.shape)))
        elif name in ("n_seqs", "max_blocks") and name in self.__dict__:
            raise AttributeError("%s is the size of the batch's tensors" % name)
        elif name == "workspace" and not value.is_contiguous():
            raise ValueError("workspace must be contiguous")
        object.__setattr__(self, name, value)
        if name == "workspace":
            # It is ready in the order of the stream that was current when a batch first took it; _use_on adds others.
            # (Another batch's workspace comes with its mark.)
            if not hasattr(value, "_ready_on"):
                made_on = torch.cuda.current_stream(value.device)
                value.record_stream(made_on)  # it may have been made elsewhere
                with torch.cuda.stream(made_on):
                    ready = None if torch.cuda.is_current_stream_capturing() else made_on.record_event()
                value._ready_on = made_on.cuda_stream, ready
            raw, self._ready = value._ready_on
            self._streams = {raw}

    def _use_on(self, raw):
        """Orders the workspace's fill before, and its release after, the calls on another stream.  (A stream under
        capture cannot wait for what was not captured with it; a graph is replayed after the work before its capture.)"""
        stream = _stream_object(raw, self.workspace.device)
        self.workspace.record_stream(stream)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        if self._ready is not None:
            stream.wait_event(self._ready)
        self._streams.add(raw)

    def same_device(self, index):
        if self._index != index:
            raise ValueError("the batch is on cuda:%d, the pools on cuda:%d" % (self._index, index))

    def pool(self, k_pages, v_pages):
        """(kv_dim, num_pages) of two pools [num_pages * page_rows, kv_dim]."""
        shape = k_pages.shape
        if shape != v_pages.shape or len(shape) != 2 or shape[0] % self.page_rows or \
                not k_pages.is_contiguous() or not v_pages.is_contiguous():
            raise ValueError("k_pages and v_pages must be contiguous [num_pages * page_rows, kv_dim] pools")
        return shape[1], shape[0] // self.page_rows


def append_paged(batch, k_new, v_new, k_pages, v_pages, q=None, q_out=None, table=None, rot_dim=None,
                 interleaved=False, stream=None):
    """Write the batch's new K (turned by `table`, when given) and V rows into the pages; with q, also
    return it turned, in the cache's type (in q_out when given; else rows that are not written are zeros)."""
    kv_dim, num_pages = batch.pool(k_pages, v_pages)
    D, G = batch.head_dim, batch.num_kv_heads
    rows, columns, ks = _rows2d(k_new, "k_new")
    v_rows, v_columns, vs = _rows2d(v_new, "v_new")
    if columns != G * D or v_columns != columns or v_rows != rows:
        raise ValueError("k_new and v_new must be [rows, %d]" % (G * D))
    dtype, cache = k_new.dtype, k_pages.dtype
    code, cache_code = _code(k_new, "k_new"), _code(k_pages, "k_pages")
    _like(dtype, "v_new", v_new)
    _like(cache, "v_pages", v_pages)
    if rot_dim is None:
        rot_dim = D
    tab, tab_rows = _table(table, rot_dim)
    index = k_pages.get_device()
    H = qs = qos = 0
    q_ptr = qo_ptr = None
    if q is not None:
        H = batch.num_heads
        q_rows, q_columns, qs = _rows2d(q, "q")
        if q_rows != rows or q_columns != H * D:
            raise ValueError("q must be [%d, %d]" % (rows, H * D))
        _like(dtype, "q", q)
        if q_out is None:
            q_out = _new(torch.zeros, (rows, H * D), cache, q.device, stream)
            qos = H * D
        else:
            o_rows, o_columns, qos = _rows2d(q_out, "q_out")
            if o_rows != rows or o_columns != q_columns:
                raise ValueError("q_out must have the shape of q")
            _like(cache, "q_out", q_out)
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
        _same_device(index, q, q_out)
    _same_device(index, v_pages, k_new, v_new, table)
    batch.same_device(index)
    _run("attn_append_paged", B.load_library().attn_append_paged, index, _handle(stream, index),
         (q_ptr, qo_ptr, k_new.data_ptr(), v_new.data_ptr(), code, k_pages.data_ptr(), v_pages.data_ptr(), cache_code,
          batch.block_table.data_ptr(), batch.q_start.data_ptr(), batch.kv_len.data_ptr(), rows, batch.n_seqs, H, G, D,
          kv_dim, qs, qos, ks, vs, batch.page_rows, num_pages, batch.max_blocks,
          rot_dim if tab is not None else 0, 1 if interleaved else 0, tab, tab_rows))
    return q_out


_CODE8 = tuple(t for t in (torch.uint8, getattr(torch, "float8_e4m3fn", None)) if t is not None)
_SCALE8 = tuple(t for t in (torch.uint8, getattr(torch, "float8_e8m0fnu", None)) if t is not None)


class PagedCache8:
    """A paged cache in 8 bits: pools of e4m3 codes and their scales (see attn_append_paged8 in attn_gqa.h).

    k_pages, v_pages [num_pages * page_rows, kv_dim] (uint8 or float8_e4m3fn) and k_scales, v_scales
    [num_pages * page_rows / scale_rows, num_kv_heads] (uint8 or float8_e8m0fnu), contiguous CUDA tensors, kept;
    PagedCache8.empty makes them."""

    __slots__ = ("k_pages", "v_pages", "k_scales", "v_scales", "rows", "kv_dim", "num_kv_heads", "scale_rows", "index")

    def __init__(self, k_pages, v_pages, k_scales, v_scales):
        for name, x, types in (("k_pages", k_pages, _CODE8), ("v_pages", v_pages, _CODE8),
                               ("k_scales", k_scales, _SCALE8), ("v_scales", v_scales, _SCALE8)):
            if x.dim() != 2 or x.dtype not in types or not x.is_contiguous():
                raise ValueError("%s must be a contiguous matrix of %s" % (name, " or ".join(map(str, types))))
        if k_pages.shape != v_pages.shape or k_scales.shape != v_scales.shape:
            raise ValueError("the pools, and the scales, of K and V must have one shape")
        (rows, kv_dim), (blocks, heads) = k_pages.shape, k_scales.shape
        if rows == 0 or blocks == 0 or heads == 0 or rows % blocks:
            raise ValueError("%d pool rows cannot be divided into %d blocks of scales" % (rows, blocks))
        index = k_pages.get_device()
        if index < 0:
            raise ValueError("the cache must be in device memory")
        _same_device(index, v_pages, k_scales, v_scales)
        for name, x in (("k_pages", k_pages), ("v_pages", v_pages), ("k_scales", k_scales), ("v_scales", v_scales),
                        ("rows", rows), ("kv_dim", kv_dim), ("num_kv_heads", heads), ("scale_rows", rows // blocks),
                        ("index", index)):
            object.__setattr__(self, name, x)

    def __setattr__(self, name, value):
        raise AttributeError("a cache keeps the tensors that it was made of")

    @classmethod
    def empty(cls, num_pages, page_rows, num_kv_heads, head_dim, scale_rows=16, device="cuda"):
        """A cache of zeros.  scale_rows positions of a head share a scale; it divides page_rows."""
        if scale_rows < 1 or page_rows % scale_rows:
            raise ValueError("scale_rows must divide page_rows")
        rows = num_pages * page_rows
        pools = [torch.zeros(rows, num_kv_heads * head_dim, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.full((rows // scale_rows, num_kv_heads), 127 - 14, dtype=torch.uint8, device=device)
                  for _ in range(2)]
        return cls(*pools, *scales)

    def pages(self, batch):
        """Pages of the pools, as the batch counts them."""
        page_rows = batch.page_rows
        if self.rows % page_rows or page_rows % self.scale_rows or self.num_kv_heads != batch.num_kv_heads:
            raise ValueError("the cache (%d rows, %d a scale, %d heads) does not fit the batch (%d rows a page, %d heads)"
                             % (self.rows, self.scale_rows, self.num_kv_heads, page_rows, batch.num_kv_heads))
        batch.same_device(self.index)
        return self.rows // page_rows


def append_paged8(batch, k_new, v_new, cache, q=None, q_out=None, table=None, rot_dim=None, interleaved=False,
                  q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """Write the batch's new K (normed by k_weight and turned by `table`, when given) and V rows into a PagedCache8;
    with q, also return it normed (q_weight) and turned, in q_out or in a new tensor (of q's type, bf16 for fp32;
    rows that are not written are zeros)."""
    num_pages = cache.pages(batch)
    D, G = batch.head_dim, batch.num_kv_heads
    rows, columns, ks = _rows2d(k_new, "k_new")
    v_rows, v_columns, vs = _rows2d(v_new, "v_new")
    if columns != G * D or v_columns != columns or v_rows != rows:
        raise ValueError("k_new and v_new must be [rows, %d]" % (G * D))
    dtype = k_new.dtype
    code = q_code = _code(k_new, "k_new")
    _like(dtype, "v_new", v_new)
    if rot_dim is None:
        rot_dim = D
    tab, tab_rows = _table(table, rot_dim)
    w_code, wq, wk = _weights(D, q_weight, k_weight)
    index = cache.index
    H = qs = qos = 0
    if q is not None:
        H = batch.num_heads
        q_rows, q_columns, qs = _rows2d(q, "q")
        if q_rows != rows or q_columns != H * D:
            raise ValueError("q must be [%d, %d]" % (rows, H * D))
        _like(dtype, "q", q)
        if q_out is None:
            q_out = _new(torch.zeros, (rows, H * D), torch.bfloat16 if dtype == torch.float32 else dtype, q.device,
                         stream)
            qos = H * D
        else:
            o_rows, o_columns, qos = _rows2d(q_out, "q_out")
            if o_rows != rows or o_columns != q_columns:
                raise ValueError("q_out must have the shape of q")
        q_code = _code(q_out, "q_out")
        _same_device(index, q, q_out)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    _same_device(index, k_new, v_new, table, q_weight, k_weight)
    _run("attn_append_paged8", B.load_library().attn_append_paged8, index, _handle(stream, index),
         (_ptr(q), _ptr(q_out), k_new.data_ptr(), v_new.data_ptr(), code, q_code, cache.k_pages.data_ptr(),
          cache.v_pages.data_ptr(), cache.k_scales.data_ptr(), cache.v_scales.data_ptr(), batch.block_table.data_ptr(),
          batch.q_start.data_ptr(), batch.kv_len.data_ptr(), rows, batch.n_seqs, H, G, D, cache.kv_dim, qs, qos, ks, vs,
          batch.page_rows, num_pages, batch.max_blocks, cache.scale_rows, wq, wk, w_code, eps,
          rot_dim if tab is not None else 0, 1 if interleaved else 0, tab, tab_rows))
    return q_out


def read_paged8(batch, cache, starts, k_out, v_out, first=None, stream=None):
    """Positions of the batch's sequences back from a PagedCache8: rows [starts[s], starts[s+1]) of k_out and v_out
    (fp32, bf16 or fp16, [rows, G*D]) become positions first[s] (None: 0), first[s] + 1, ...  starts [n + 1] and
    first [n] are int32 CUDA tensors.  Rows of no sequence are left as they are.  Returns (k_out, v_out)."""
    num_pages = cache.pages(batch)
    G, D = batch.num_kv_heads, batch.head_dim
    rows, columns, ks = _rows2d(k_out, "k_out")
    v_rows, v_columns, vs = _rows2d(v_out, "v_out")
    if columns != G * D or v_columns != columns or v_rows != rows:
        raise ValueError("k_out and v_out must be [rows, %d]" % (G * D))
    code = _code(k_out, "k_out")
    _like(k_out.dtype, "v_out", v_out)
    if starts.shape != (batch.n_seqs + 1,) or (first is not None and first.shape != (batch.n_seqs,)):
        raise ValueError("starts must hold %d entries and first %d" % (batch.n_seqs + 1, batch.n_seqs))
    index = cache.index
    _same_device(index, k_out, v_out, starts, first)
    _run("attn_read_paged8", B.load_library().attn_read_paged8, index, _handle(stream, index),
         (cache.k_pages.data_ptr(), cache.v_pages.data_ptr(), cache.k_scales.data_ptr(), cache.v_scales.data_ptr(),
          k_out.data_ptr(), v_out.data_ptr(), code, batch.block_table.data_ptr(), _int32(starts, "starts"),
          _int32(first, "first"), batch.kv_len.data_ptr(), rows, batch.n_seqs, G, D, cache.kv_dim, ks, vs,
          batch.page_rows, num_pages, batch.max_blocks, cache.scale_rows))
    return k_out, v_out


def _attend_args(batch, q, out, cache_type, scale, window, sinks, alibi_slopes, prefix_len, stream):
    """What attend_paged and attend_paged8 check alike: (type code, rows, q stride, out, out stride, scale, slopes)."""
    H, D = batch.num_heads, batch.head_dim
    rows, columns, qs = _rows2d(q, "q")
    if columns != H * D:
        raise ValueError("q must be [rows, %d]" % (H * D))
    dtype = q.dtype
    code = _code(q, "q")
    if cache_type is not None and cache_type != dtype:
        raise ValueError("k_pages has type %s, unlike the tensors it goes with (%s)" % (cache_type, dtype))
    if out is None:
        out = _new(torch.zeros, (rows, H * D), dtype, q.device, stream)
        os = H * D
    else:
        out_rows, out_columns, os = _rows2d(out, "out")
        if out_rows != rows or out_columns != columns:
            raise ValueError("out must have the shape of q")
        _like(dtype, "out", out)
    slopes = None
    if alibi_slopes is not None:
        if alibi_slopes.numel() != H or alibi_slopes.dtype != torch.float32 or not alibi_slopes.is_contiguous():
            raise ValueError("alibi_slopes must hold one float32 slope a head")
        slopes = alibi_slopes.data_ptr()
    if prefix_len is not None and prefix_len.numel() != batch.n_seqs:
        raise ValueError("prefix_len must hold one length a sequence")
    if window or sinks:
        _count32("window", window)
        _count32("sinks", sinks)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    return code, rows, qs, out, os, scale, slopes


def _attend_stream(batch, index, stream):
    batch.same_device(index)
    stream = _handle(stream, index)
    if stream not in batch._streams:
        batch._use_on(stream)
    return stream


def attend_paged(batch, q, k_pages, v_pages, out=None, scale=None, window=0, softcap=0.0, alibi_slopes=None,
                 prefix_len=None, stream=None, sinks=0):
    """Attention of the batch's new tokens, q [rows, H*D] (bf16 or fp16), over its pages: the last `window`
    keys of each row (0 = all) and its sequence's first `sinks`, scores capped by softcap * tanh(s / softcap) (0 =
    uncapped) and biased by -alibi_slopes[h] * distance, keys below prefix_len[s] visible to every row.  Rows of no
    sequence are left as they are in `out`."""
    kv_dim, num_pages = batch.pool(k_pages, v_pages)
    code, rows, qs, out, os, scale, slopes = _attend_args(batch, q, out, k_pages.dtype, scale, window, sinks,
                                                          alibi_slopes, prefix_len, stream)
    _like(q.dtype, "v_pages", v_pages)
    index = k_pages.get_device()
    workspace = batch.workspace
    _same_device(index, v_pages, q, out, alibi_slopes, prefix_len, workspace)
    _run("attn_batch_paged_sinks" if sinks else "attn_batch_paged", B.load_library().attn_batch_paged_sinks, index,
         _attend_stream(batch, index, stream),
         (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), code,
          batch.block_table.data_ptr(), batch.q_start.data_ptr(), batch.kv_len.data_ptr(), rows, batch.n_seqs,
          batch.num_heads, batch.num_kv_heads, batch.head_dim, kv_dim, qs, os, batch.page_rows, num_pages,
          batch.max_blocks, scale, window, softcap, slopes, _int32(prefix_len, "prefix_len"), workspace.data_ptr(),
          workspace.numel(), sinks))
    return out


def attend_paged8(batch, q, cache, out=None, scale=None, window=0, sinks=0, softcap=0.0, alibi_slopes=None,
                  prefix_len=None, stream=None):
    """attend_paged over a PagedCache8; q and out are bf16 or fp16."""
    num_pages = cache.pages(batch)
    code, rows, qs, out, os, scale, slopes = _attend_args(batch, q, out, None, scale, window, sinks, alibi_slopes,
                                                          prefix_len, stream)
    index = cache.index
    workspace = batch.workspace
    _same_device(index, q, out, alibi_slopes, prefix_len, workspace)
    _run("attn_batch_paged8", B.load_library().attn_batch_paged8, index, _attend_stream(batch, index, stream),
         (q.data_ptr(), cache.k_pages.data_ptr(), cache.v_pages.data_ptr(), cache.k_scales.data_ptr(),
          cache.v_scales.data_ptr(), out.data_ptr(), code, batch.block_table.data_ptr(), batch.q_start.data_ptr(),
          batch.kv_len.data_ptr(), rows, batch.n_seqs, batch.num_heads, batch.num_kv_heads, batch.head_dim,
          cache.kv_dim, qs, os, batch.page_rows, num_pages, batch.max_blocks, cache.scale_rows, scale, window, sinks,
          softcap, slopes, _int32(prefix_len, "prefix_len"), workspace.data_ptr(), workspace.numel()))
    return out
