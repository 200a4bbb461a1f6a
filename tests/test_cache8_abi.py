"""Refusals of the head norms and of the 8-bit paged cache, without a GPU (as
test_batch_abi.py: made-up device addresses that host validation must refuse
before anything is launched)."""
import os
import subprocess
import sys

import pytest

from test_abi import FAKE, ROOT, gpu_visible

hidden = pytest.mark.skipif(gpu_visible(), reason="a GPU is visible: runs in a child process with the device hidden")
BAD, UNSUP = 1, 2
P = [FAKE + 0x1000 * i for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    from attention_gqa_online_gb300 import build
    build.build()
    import attention_gqa_online_gb300 as A
    return A.load_library()


def norm_call(lib, q=P[0], k=P[1], qo=P[2], ko=P[3], wq=P[4], wk=P[5], dt=1, wdt=1, rows=4, H=4, G=2, D=64, qs=256,
              ks=128, qos=256, kos=128, eps=1e-6, R=64, layout=0, pos=P[6], table=P[7], trows=16):
    return lib.attn_qk_norm_rope(q, k, qo, ko, wq, wk, dt, wdt, rows, H, G, D, qs, ks, qos, kos, eps, R, layout, pos,
                                 table, trows, None)


NORM_BAD = [
    dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(dt=3), dict(dt=-1), dict(wdt=3), dict(H=0, G=0),
    dict(H=2 ** 21, qs=2 ** 28, qos=2 ** 28), dict(D=0), dict(D=258, qs=2048, ks=2048, qos=2048, kos=2048), dict(R=63),
    dict(R=66), dict(table=None), dict(table=P[7] + 2), dict(pos=P[6] + 2), dict(pos=None, trows=3), dict(qs=255),
    dict(ks=127), dict(qos=255), dict(kos=127), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(eps=1e-31), dict(layout=2), dict(q=P[0] + 1), dict(wk=P[5] + 1),
    dict(wdt=0, wq=P[4] + 2), dict(dt=0, ko=P[3] + 2), dict(qo=P[0], qos=264), dict(ko=P[1], kos=264)]


@hidden
@pytest.mark.parametrize("kw", NORM_BAD)
def test_norm_rejects(lib, kw):
    assert norm_call(lib, **kw) == BAD


def norm_back(lib, dq=P[8], dk=P[9], dwq=P[10], dwk=P[11], dqs=256, dks=128, ws=FAKE, wsb=1 << 30, q=P[0], k=P[1],
              qo=P[2], ko=P[3], wq=P[4], wk=P[5], dt=1, wdt=1, rows=4, H=4, G=2, D=64, qs=256, ks=128, qos=256, kos=128,
              eps=1e-6, R=64, layout=0, pos=P[6], table=P[7], trows=16):
    return lib.attn_qk_norm_rope_backward(dq, dk, q, k, qo, ko, wq, wk, dwq, dwk, dt, wdt, rows, H, G, D, dqs, dks, qs,
                                          ks, qos, kos, eps, R, layout, pos, table, trows, ws, wsb, None)


@hidden
@pytest.mark.parametrize("kw", NORM_BAD + [
    dict(dq=None), dict(dk=None), dict(dqs=255), dict(dks=127), dict(dq=P[8] + 1), dict(dwk=P[11] + 1),
    dict(qo=P[8], qos=264), dict(ko=P[9], kos=264)])
def test_norm_backward_rejects(lib, kw):
    assert norm_back(lib, **kw) == BAD


@hidden
def test_norm_of_no_rows_is_noop(lib):
    none = dict(rows=0, q=None, k=None, qo=None, ko=None)
    assert norm_call(lib, **none) == 0
    assert norm_back(lib, dq=None, dk=None, dwq=None, dwk=None, ws=None, wsb=0, **none) == 0
    assert lib.attn_qk_norm_rope_backward_workspace_bytes(0) == 0
    assert lib.attn_qk_norm_rope_backward_workspace_bytes(257) == 0


def append_call(lib, q=P[0], qo=P[1], k=P[2], v=P[3], dt=1, qdt=1, kp=P[4], vp=P[5], ks=P[6], vs=P[7], bt=P[8], qst=P[9],
                kvl=P[10], rows=4, n=2, H=4, G=2, D=64, kvd=128, qs=256, qos=256, kstr=128, vstr=128, pr=16, np=8, mb=4,
                sr=8, wq=FAKE, wk=FAKE, wdt=1, eps=1e-6, R=64, layout=0, table=P[11], trows=16):
    return lib.attn_append_paged8(q, qo, k, v, dt, qdt, kp, vp, ks, vs, bt, qst, kvl, rows, n, H, G, D, kvd, qs, qos,
                                  kstr, vstr, pr, np, mb, sr, wq, wk, wdt, eps, R, layout, table, trows, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(ks=None), dict(vs=None),
    dict(bt=None), dict(qst=None), dict(kvl=None), dict(dt=3), dict(qdt=0), dict(qdt=3), dict(wdt=3), dict(layout=2),
    dict(H=0), dict(q=None, qo=None, H=0), dict(G=0), dict(D=0), dict(D=144, kvd=1024, qs=1024, qos=1024, kstr=1024, vstr=1024),
    dict(kvd=127), dict(qs=255), dict(qos=255), dict(kstr=127), dict(vstr=127), dict(pr=0), dict(np=0), dict(mb=0),
    dict(sr=0), dict(sr=3), dict(sr=32), dict(np=2 ** 28), dict(mb=2 ** 28), dict(rows=2 ** 31), dict(n=2 ** 30 + 1),
    dict(R=63), dict(R=66), dict(table=None), dict(trows=0), dict(table=P[11] + 2), dict(eps=0.0), dict(eps=float("nan")),
    dict(k=P[2] + 1), dict(qo=P[1] + 1), dict(kvl=P[10] + 2), dict(wk=FAKE + 1), dict(q=P[1], qos=264),
    dict(q=P[1], dt=0, k=P[2], qdt=2)])
def test_append_rejects(lib, kw):
    assert append_call(lib, **kw) == BAD


@hidden
@pytest.mark.parametrize("kw", [
    dict(dt=1, qdt=2), dict(dt=2, qdt=1, wdt=2), dict(D=24, kvd=128, R=24), dict(kvd=136), dict(kp=P[4] + 8), dict(vp=P[5] + 8)])
def test_append_unsupported(lib, kw):
    assert append_call(lib, **kw) == UNSUP


@hidden
def test_append_of_nothing_is_noop(lib):
    for kw in (dict(rows=0), dict(n=0)):
        assert append_call(lib, k=None, v=None, kp=None, vp=None, **kw) == 0


def read_call(lib, kp=P[0], vp=P[1], ks=P[2], vs=P[3], ko=P[4], vo=P[5], dt=1, bt=P[6], st=P[7], first=P[8], kvl=P[9],
              rows=4, n=2, G=2, D=64, kvd=128, kstr=128, vstr=128, pr=16, np=8, mb=4, sr=8):
    return lib.attn_read_paged8(kp, vp, ks, vs, ko, vo, dt, bt, st, first, kvl, rows, n, G, D, kvd, kstr, vstr, pr, np,
                                mb, sr, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(kp=None), dict(vp=None), dict(ks=None), dict(vs=None), dict(ko=None), dict(vo=None), dict(bt=None),
    dict(st=None), dict(kvl=None), dict(dt=3), dict(G=0), dict(D=0), dict(D=144, kvd=1024, kstr=1024, vstr=1024),
    dict(kvd=127), dict(kstr=127), dict(vstr=127), dict(pr=0), dict(np=0), dict(mb=0), dict(sr=0), dict(sr=5),
    dict(np=2 ** 28), dict(rows=2 ** 31), dict(n=2 ** 30 + 1), dict(ko=P[4] + 1), dict(dt=0, vo=P[5] + 2),
    dict(st=P[7] + 2), dict(first=P[8] + 2)])
def test_read_rejects(lib, kw):
    assert read_call(lib, **kw) == BAD


@hidden
@pytest.mark.parametrize("kw", [dict(D=24, kvd=128), dict(kvd=136), dict(kp=P[0] + 8), dict(vp=P[1] + 8)])
def test_read_unsupported(lib, kw):
    assert read_call(lib, **kw) == UNSUP


@hidden
def test_read_of_nothing_is_noop(lib):
    for kw in (dict(rows=0), dict(n=0)):
        assert read_call(lib, kp=None, ko=None, st=None, **kw) == 0


def test_python_layer_refuses_host_tensors_and_shapes_that_do_not_fit(lib):
    import torch

    import attention_gqa_online_gb300 as A
    q, k, w = torch.zeros(4, 128), torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="device memory"):
        A.qk_norm_rope(q, k, 2, 1, w, w)
    with pytest.raises(ValueError, match="device memory"):
        A.qk_norm_rope_backward(q, k, q, k, 2, 1, w, w)
    for bad in (dict(k=torch.zeros(3, 64)), dict(k=torch.zeros(4, 32)), dict(k=k.half()), dict(q_weight=torch.ones(32)),
                dict(q_weight=w.half()), dict(rot_dim=64), dict(positions=torch.zeros(4, dtype=torch.int64)),
                dict(table=torch.zeros(4, 32)), dict(positions=torch.zeros(3, dtype=torch.int32)), dict(q=q[:, ::2]),
                dict(q_out=torch.zeros(4, 64)), dict(q_out=q.half()), dict(num_heads=3)):
        with pytest.raises(ValueError):
            A.qk_norm_rope(**dict(dict(q=q, k=k, num_heads=2, num_kv_heads=1, q_weight=w, k_weight=w), **bad))
    with pytest.raises(ValueError, match="shape of q"):
        A.qk_norm_rope_backward(q[:3], k, q, k, 2, 1, w, w)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError, match="device memory"):
        A.PagedCache8(u8(16, 32), u8(16, 32), u8(4, 2), u8(4, 2))
    for bad in ((u8(16, 32).float(), u8(16, 32), u8(4, 2), u8(4, 2)), (u8(16, 32), u8(8, 32), u8(4, 2), u8(4, 2)),
                (u8(16, 32), u8(16, 32), u8(3, 2), u8(3, 2)), (u8(16, 32), u8(16, 32), u8(4, 2), u8(4, 1)),
                (u8(16, 64)[:, ::2], u8(16, 32), u8(4, 2), u8(4, 2)), (u8(0, 32), u8(0, 32), u8(0, 2), u8(0, 2)),
                (u8(16, 32), u8(16, 32), u8(4, 2).int(), u8(4, 2).int())):
        with pytest.raises(ValueError):
            A.PagedCache8(*bad)
    with pytest.raises(ValueError, match="divide"):
        A.PagedCache8.empty(2, 16, 2, 16, scale_rows=5, device="cpu")


def test_refusals_run_with_the_device_hidden():
    if not gpu_visible():
        pytest.skip("ran above")
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", os.path.abspath(__file__)], env=env, cwd=ROOT,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def attend_call(lib, q=P[0], kp=P[1], vp=P[2], ks=P[3], vs=P[4], out=P[5], dt=1, bt=P[6], st=P[7], kvl=P[8], rows=4, n=2,
                H=4, G=2, D=64, kvd=128, qs=256, os=256, pr=16, np=8, mb=4, sr=8, scale=0.1, window=0, sinks=0, cap=0.0,
                slopes=P[9], prefix=P[10], ws=P[11], wsb=1 << 40):
    return lib.attn_batch_paged8(q, kp, vp, ks, vs, out, dt, bt, st, kvl, rows, n, H, G, D, kvd, qs, os, pr, np, mb, sr,
                                 scale, window, sinks, cap, slopes, prefix, ws, wsb, None)


@hidden
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(kp=None), dict(vp=None), dict(ks=None), dict(vs=None), dict(out=None), dict(bt=None),
    dict(st=None), dict(kvl=None), dict(dt=3), dict(H=0), dict(G=0), dict(H=5), dict(D=0),
    dict(D=144, kvd=1024, qs=1024, os=1024), dict(kvd=127), dict(qs=255), dict(os=255), dict(pr=0), dict(np=0),
    dict(mb=0), dict(sr=0), dict(sr=3), dict(sr=32), dict(scale=float("nan")), dict(scale=3e38), dict(cap=-1.0),
    dict(cap=float("inf")), dict(bt=P[6] + 2), dict(slopes=P[9] + 1), dict(prefix=P[10] + 2)])
def test_attend_rejects(lib, kw):
    assert attend_call(lib, **kw) == BAD


@hidden
@pytest.mark.parametrize("kw", [
    dict(dt=0), dict(D=24, kvd=128), dict(kvd=136), dict(qs=260), dict(os=260), dict(q=P[0] + 8), dict(kp=P[1] + 8),
    dict(vp=P[2] + 8), dict(out=P[5] + 8), dict(n=16385), dict(mb=2 ** 21), dict(rows=2 ** 29)])
def test_attend_unsupported(lib, kw):
    assert attend_call(lib, **kw) == UNSUP


@hidden
def test_attend_of_nothing_is_noop(lib):
    for kw in (dict(rows=0), dict(n=0)):
        assert attend_call(lib, q=None, ks=None, **kw) == 0


@hidden
def test_append_of_no_rows_with_queries_is_noop(lib):
    """Tensors of no rows have no address."""
    for kw in (dict(rows=0), dict(n=0)):
        assert append_call(lib, q=None, qo=None, k=None, v=None, **kw) == 0
