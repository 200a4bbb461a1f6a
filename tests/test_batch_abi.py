"""Refusals of the rotary operator and the batched paged calls, without a GPU.

As in test_abi.py, the calls pass made-up device addresses that host
validation must refuse before anything is launched, so they run only where no
GPU is visible; elsewhere the last test runs this module in a child process
with the device hidden."""
import math
import os
import subprocess
import sys

import pytest

from test_abi import FAKE, ROOT, gpu_visible

hidden = pytest.mark.skipif(gpu_visible(), reason="a GPU is visible: runs in a child process with the device hidden")
BAD, UNSUP = 1, 2


@pytest.fixture(scope="module")
def lib():
    from attention_gqa_online_gb300 import build
    build.build()
    import attention_gqa_online_gb300 as A
    return A.load_library()


def table_call(lib, table=FAKE, rows=8, R=64, base=1e4, kind=0, f=4.0, orig=2048, fast=32.0, slow=1.0, m=1.0):
    return lib.attn_rope_table_scaled(table, rows, R, base, kind, f, orig, fast, slow, m, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(R=0), dict(R=7), dict(R=1026), dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(kind=4),
    dict(kind=-1), dict(kind=1, f=0.0), dict(kind=2, f=-1.0), dict(kind=3, f=math.inf), dict(kind=2, R=2),
    dict(kind=3, orig=0), dict(kind=3, fast=1.0, slow=1.0), dict(kind=3, slow=math.nan), dict(m=math.nan),
    dict(table=None), dict(table=FAKE + 2), dict(rows=2 ** 26),
])
def test_scaled_table_rejects(lib, kw):
    assert table_call(lib, **kw) == BAD


@hidden
def test_scaled_table_of_no_rows_is_noop(lib):
    assert table_call(lib, table=None, rows=0) == 0


def rope_call(lib, x=FAKE, y=FAKE + 0x1000, dt=1, rows=4, heads=2, D=64, R=64, xs=128, ys=128, layout=0, pos=FAKE,
              table=FAKE, trows=16, inv=0):
    return lib.attn_rope_apply(x, y, dt, rows, heads, D, R, xs, ys, layout, pos, table, trows, inv, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(x=None), dict(y=None), dict(table=None), dict(dt=3), dict(dt=-1), dict(layout=2), dict(heads=0), dict(D=0),
    dict(D=1025, xs=4096, ys=4096), dict(R=0), dict(R=63), dict(R=66), dict(xs=127), dict(ys=127),
    dict(y=FAKE, ys=136), dict(pos=None, trows=3), dict(x=FAKE + 1), dict(dt=0, x=FAKE + 2), dict(table=FAKE + 2),
    dict(pos=FAKE + 1), dict(heads=2 ** 31, xs=2 ** 32 - 1, ys=2 ** 32 - 1),
])
def test_rope_apply_rejects(lib, kw):
    assert rope_call(lib, **kw) == BAD


@hidden
def test_rope_apply_of_no_rows_is_noop(lib):
    assert rope_call(lib, x=None, y=None, table=None, pos=None, rows=0) == 0


def append_call(lib, q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, dt=1, kp=FAKE, vp=FAKE, cdt=1, bt=FAKE, qs=FAKE, kl=FAKE,
                rows=4, n=2, H=4, G=2, D=64, kv_dim=128, q_stride=256, qo_stride=256, k_stride=128, v_stride=128,
                page_rows=16, pages=8, blocks=4, R=64, layout=0, table=FAKE, trows=64):
    return lib.attn_append_paged(q, q_out, k, v, dt, kp, vp, cdt, bt, qs, kl, rows, n, H, G, D, kv_dim, q_stride,
                                 qo_stride, k_stride, v_stride, page_rows, pages, blocks, R, layout, table, trows, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(qs=None), dict(kl=None),
    dict(q=None), dict(H=0), dict(q_out=None), dict(H=5), dict(G=0), dict(D=0), dict(D=129), dict(dt=3), dict(cdt=-1),
    dict(layout=2), dict(kv_dim=127), dict(q_stride=255), dict(qo_stride=255), dict(k_stride=127), dict(v_stride=127),
    dict(page_rows=0), dict(pages=0), dict(blocks=0), dict(page_rows=2 ** 20, blocks=2 ** 11), dict(R=63), dict(R=66),
    dict(table=None), dict(trows=0), dict(k=FAKE + 1), dict(kp=FAKE + 1), dict(bt=FAKE + 2), dict(rows=2 ** 31),
    dict(n=2 ** 31),
])
def test_append_rejects(lib, kw):
    assert append_call(lib, **kw) == BAD


@hidden
@pytest.mark.parametrize("dt,cdt", [(1, 0), (1, 2), (2, 0), (2, 1)])
def test_append_rejects_type_pairs(lib, dt, cdt):
    assert append_call(lib, dt=dt, cdt=cdt) == UNSUP


@hidden
@pytest.mark.parametrize("kw", [dict(qo_stride=264), dict(dt=0, cdt=1)])
def test_append_rejects_q_in_place_in_another_layout(lib, kw):
    assert append_call(lib, rows=4, k=FAKE + 0x1000, **kw) == BAD


@hidden
def test_append_of_nothing_is_noop(lib):
    assert append_call(lib, rows=0, k=None, v=None, bt=None) == 0
    assert append_call(lib, n=0, qs=None, kl=None) == 0


def batch_call(lib, q=FAKE, kp=FAKE, vp=FAKE, out=FAKE, dt=1, bt=FAKE, qs=FAKE, kl=FAKE, rows=4, n=2, H=4, G=2, D=64,
               kv_dim=128, q_stride=256, o_stride=256, page_rows=16, pages=8, blocks=4, scale=0.125, window=0, cap=0.0,
               slopes=None, prefix=None, ws=FAKE, nbytes=1 << 30):
    return lib.attn_batch_paged(q, kp, vp, out, dt, bt, qs, kl, rows, n, H, G, D, kv_dim, q_stride, o_stride,
                                page_rows, pages, blocks, scale, window, cap, slopes, prefix, ws, nbytes, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(kp=None), dict(vp=None), dict(out=None), dict(bt=None), dict(qs=None), dict(kl=None),
    dict(H=5), dict(G=0), dict(D=0), dict(D=136), dict(dt=3), dict(kv_dim=120), dict(q_stride=248),
    dict(o_stride=248), dict(page_rows=0), dict(pages=0), dict(blocks=0), dict(page_rows=2 ** 16, pages=2 ** 15),
    dict(scale=math.inf), dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.inf), dict(cap=math.nan),
    dict(bt=FAKE + 2), dict(qs=FAKE + 1), dict(kl=FAKE + 2), dict(slopes=FAKE + 2), dict(prefix=FAKE + 2),
])
def test_batch_rejects(lib, kw):
    assert batch_call(lib, **kw) == BAD


@hidden
@pytest.mark.parametrize("kw", [
    dict(dt=0), dict(D=60, kv_dim=128), dict(kv_dim=132), dict(q_stride=260), dict(o_stride=260), dict(q=FAKE + 2),
    dict(kp=FAKE + 8), dict(vp=FAKE + 8), dict(out=FAKE + 8), dict(n=16385), dict(rows=2 ** 29),
    dict(page_rows=2 ** 14, blocks=2 ** 11, pages=8),
])
def test_batch_unsupported(lib, kw):
    assert batch_call(lib, **kw) == UNSUP


@hidden
def test_batch_of_nothing_is_noop(lib):
    assert batch_call(lib, rows=0, q=None, out=None) == 0
    assert batch_call(lib, n=0, qs=None, kl=None, bt=None) == 0


@hidden
def test_batch_workspace_rejects_bad_heads(lib):
    assert lib.attn_batch_paged_workspace_bytes(5, 2, 64) == 0
    assert lib.attn_batch_paged_workspace_bytes(4, 0, 64) == 0
    assert lib.attn_batch_paged_workspace_bytes(4, 2, 0) == 0
    assert lib.attn_batch_paged_workspace_bytes(4, 2, 129) == 0


@hidden
def test_python_layer_refuses_host_tensors_and_mismatched_types(lib):
    import torch
    import attention_gqa_online_gb300 as A
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be in device memory"):
        A.attn_rope_apply(x, x, 4, 2, 64, 64, 128, 128, 0, None, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="unlike the tensors"):
        A.attn_rope_apply(x, x.float(), 4, 2, 64, 64, 128, 128, 0, None, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        A.attn_rope_apply(x.double(), x, 4, 2, 64, 64, 128, 128, 0, None, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="not a multiple"):
        A.rope(x, torch.zeros(4, 64), 3)
    with pytest.raises(ValueError, match="table must be"):
        A.rope(x, torch.zeros(4, 64), 2, rot_dim=32)
    with pytest.raises(ValueError, match="one position a row"):
        A.rope(x, torch.zeros(4, 64), 2, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous columns"):
        A.rope(torch.zeros(128, 4).t(), torch.zeros(4, 64), 2)
    with pytest.raises(ValueError, match="do not fit together"):
        A.PagedBatch(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                     torch.zeros(2, dtype=torch.int32), 4, 2, 64, 16)


@hidden
@pytest.mark.parametrize("kw", [dict(cap=1e-38, scale=10.0), dict(cap=1e-38, scale=-10.0), dict(cap=3e38)])
def test_batch_rejects_caps_outside_the_range_of_its_arithmetic(lib, kw):
    """scale / softcap and softcap log2 e have to be finite."""
    assert batch_call(lib, **kw) == BAD


@hidden
@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_batch_rejects_scales_outside_the_range_of_its_arithmetic(lib, scale):
    """scale log2 e has to be finite: infinite, it would make NaN of zero scores."""
    assert batch_call(lib, scale=scale) == BAD


@hidden
def test_batch_refuses_pools_whose_last_boxes_pass_31_bits(lib):
    assert batch_call(lib, page_rows=2 ** 8, pages=2 ** 23 - 1) == UNSUP


@hidden
def test_python_layer_refuses_sizes_that_do_not_fit_32_bits(lib):
    """Tensors without memory behind them."""
    import torch
    import attention_gqa_online_gb300 as A
    table = torch.zeros(4, 2)
    for shape, strides in (((2 ** 32 + 1, 2), (2, 1)), ((2, 2), (2 ** 32 + 2, 1))):
        x = torch.empty_strided(shape, strides, dtype=torch.bfloat16, device="meta")
        with pytest.raises(ValueError, match="32 bits"):
            A.rope(x, table, 1)


@hidden
@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 32, 2 ** 31 - 1])
def test_append_rejects_counts_that_its_search_cannot_add_to(lib, n):
    """The search of a row's sequence rounds up n_seqs / 32 in 32-bit arithmetic."""
    assert append_call(lib, n=n, k=FAKE + 0x1000) == BAD


@hidden
@pytest.mark.parametrize("value", [2 ** 32, 2 ** 32 + 5, -1])
def test_python_layer_refuses_counts_that_would_wrap_in_32_bits(lib, value):
    """ctypes keeps the low 32 bits of what it is given: a window of 2^32 + 5 became one of 5."""
    import torch
    import attention_gqa_online_gb300 as A
    b = object.__new__(A.PagedBatch)
    for name, x in dict(_index=-1, n_seqs=1, max_blocks=1, num_heads=1, num_kv_heads=1, head_dim=8, page_rows=8).items():
        object.__setattr__(b, name, x)
    q, pool = torch.zeros(1, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="window"):
        A.attend_paged(b, q, pool, pool, out=q.clone(), window=value)
    with pytest.raises(ValueError, match="orig_max_pos"):
        A.rope_table(16, 64, scaling="by_parts", factor=2.0, orig_max_pos=value)


def test_the_package_imports_under_a_torch_without_cuda():
    """torch's private CUDA queries, which such a build lacks, are only a shorter way to the public ones."""
    code = ("import torch\nfor n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n    delattr(torch._C, n)\n"
            "import attention_gqa_online_gb300 as A\nprint('imported', A.api._current_device.__name__)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.split() == ["imported", "current_device"], r.stderr[-2000:]


@hidden
def test_batch_objects_keep_sizes_and_tensors_together(lib):
    """What the device reads follows from the tensors' shapes: sizes are not set apart from them.  (The object is
    made without its tensors, which would have to be in device memory.)"""
    import torch
    import attention_gqa_online_gb300 as A
    b = object.__new__(A.PagedBatch)
    for name, value in dict(_index=-1, n_seqs=2, max_blocks=3, workspace=None).items():
        object.__setattr__(b, name, value)
    i32 = dict(dtype=torch.int32)
    b.block_table, b.q_start, b.kv_len = torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    for name, value in (("n_seqs", 3), ("max_blocks", 4), ("block_table", torch.zeros(3, 2, **i32)),
                        ("block_table", torch.zeros(6, **i32)), ("q_start", torch.zeros(4, **i32)),
                        ("q_start", torch.zeros(3, 1, **i32)), ("kv_len", torch.zeros(2)),
                        ("workspace", torch.zeros(1, dtype=torch.uint8).expand(1 << 20))):
        before = getattr(b, name)
        with pytest.raises((AttributeError, ValueError)):
            setattr(b, name, value)
        assert getattr(b, name) is before


@hidden
@pytest.mark.parametrize("kw", [dict(factor=4.0), dict(orig_max_pos=4096), dict(beta_fast=16.0), dict(beta_slow=2.0),
                                dict(factor=4.0, attn_factor=1.2), dict(scaling="yarn", factor=2.0)])
def test_rope_table_refuses_what_it_would_not_use(lib, kw):
    """Values that belong to a scaling, without one, and scalings that do not exist: before memory is asked for."""
    import attention_gqa_online_gb300 as A
    with pytest.raises(ValueError, match="scaling"):
        A.rope_table(16, 64, **kw)


def test_refusals_run_with_the_device_hidden():
    if not gpu_visible():
        pytest.skip("no GPU visible: the tests above run in this process")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_batch_abi.py")], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert " passed" in r.stdout


@hidden
def test_append_of_no_rows_with_queries_is_noop(lib):
    """Tensors of no rows have no address."""
    assert append_call(lib, rows=0, q=None, q_out=None, k=None, v=None) == 0
    assert append_call(lib, n=0, q=None, q_out=None, qs=None, kl=None) == 0
