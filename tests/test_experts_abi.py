"""The gate's and the experts' entry points without a GPU: every argument error
is refused with EP_ERR_INVALID_ARG before any CUDA call."""
import ctypes

import pytest

from combine_ep_get_03_gb300 import build as cuda_build
from combine_ep_get_03_gb300 import ep

BAD = ep.EP_ERR_INVALID_ARG
P = 4096  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ep.lib()


def groups(count=P, offset=P, num=4, rows=64, per=0, status=0):
    return ep._GROUPS.pack(count, offset, num, rows, per, status)


def rows8(data=P, scales=P, row=1, group=64):
    return ep._FP8_ROWS.pack(data, scales, row, group)


def test_struct_sizes_are_the_headers():
    class Groups(ctypes.Structure):
        _fields_ = [("count", ctypes.c_void_p), ("offset", ctypes.c_void_p), ("num_groups", ctypes.c_int),
                    ("rows", ctypes.c_int64), ("rows_per_group", ctypes.c_int64), ("status", ctypes.c_void_p)]

    class Rows(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                    ("group_stride", ctypes.c_int64)]

    assert ep._GROUPS.size == ctypes.sizeof(Groups) and ep._FP8_ROWS.size == ctypes.sizeof(Rows)
    g = Groups.from_buffer_copy(ep._GROUPS.pack(1, 2, 3, 4, 5, 6))
    assert (g.count, g.offset, g.num_groups, g.rows, g.rows_per_group, g.status) == (1, 2, 3, 4, 5, 6)
    r = Rows.from_buffer_copy(ep._FP8_ROWS.pack(1, 2, 3, 4))
    assert (r.data, r.scales, r.row_stride, r.group_stride) == (1, 2, 3, 4)


def test_workspace_bytes(lib):
    n = ctypes.c_int64()
    assert lib.ep_gate_workspace_bytes(256, ctypes.byref(n)) == ep.EP_OK and n.value == 16 + 12 * 256
    for E in (0, -1, 4097):
        assert lib.ep_gate_workspace_bytes(E, ctypes.byref(n)) == BAD
    assert lib.ep_gate_workspace_bytes(8, None) == BAD


GATE = dict(logits=P, type=0, ld=64, mask=None, T=8, E=64, k=4, groups=4, keep=2, score=0, coef=0.1, idx=P, bits=64,
            w=P, count=P, prob=P, loss=P, work=P)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=P + 2), dict(type=2), dict(ld=63), dict(T=-1), dict(T=(1 << 26) + 1), dict(E=0),
    dict(E=4097, ld=5000), dict(k=0), dict(k=33), dict(k=65), dict(groups=0), dict(groups=3), dict(groups=128, E=128, ld=128),
    dict(keep=0), dict(keep=5), dict(score=2), dict(idx=None), dict(idx=P + 4), dict(bits=16), dict(w=None),
    dict(w=P + 1), dict(count=None), dict(count=P + 2), dict(prob=None), dict(loss=None), dict(work=None),
    dict(work=P + 8)])
def test_gate_forward_refusals(lib, bad):
    a = {**GATE, **bad}
    assert lib.ep_gate_forward(a["logits"], a["type"], a["ld"], a["mask"], a["T"], a["E"], a["k"], a["groups"],
                               a["keep"], a["score"], a["coef"], a["idx"], a["bits"], a["w"], a["count"], a["prob"],
                               a["loss"], a["work"], 0, None) == BAD


BACK = dict(logits=P, type=0, ld=64, T=8, E=64, k=4, score=0, idx=P, bits=64, count=P, dw=P, dl=P, out=P, old=64)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(type=-1), dict(ld=0), dict(T=-1), dict(E=0), dict(k=0), dict(score=7), dict(idx=None),
    dict(idx=P + 4), dict(bits=0), dict(count=None), dict(dw=P + 2), dict(dl=P + 1), dict(out=None), dict(out=P + 2),
    dict(old=63)])
def test_gate_backward_refusals(lib, bad):
    a = {**BACK, **bad}
    assert lib.ep_gate_backward(a["logits"], a["type"], a["ld"], None, a["T"], a["E"], a["k"], a["score"], 0.1,
                                a["idx"], a["bits"], a["count"], a["dw"], a["dl"], a["out"], a["old"], 0, None) == BAD


BAD_GROUPS = [groups(count=0), groups(count=P + 2), groups(offset=P + 1), groups(num=0), groups(num=4097),
              groups(rows=-1), groups(rows=1 << 31), groups(offset=0, per=-1), groups(offset=0, per=17),
              groups(status=P + 2), None]
BAD_ROWS = [rows8(data=0), rows8(data=P + 8), rows8(scales=0), rows8(scales=P + 2), rows8(row=-1), rows8(group=-1), None]


def test_no_rows_is_no_work(lib):
    g = groups(rows=0)
    assert lib.ep_grouped_matmul(g, None, P, P, 256, 256, None, 0, None) == ep.EP_OK
    assert lib.ep_grouped_matmul_swiglu(g, None, P, P, 256, 256, None, None, None, 0, None) == ep.EP_OK
    assert lib.ep_grouped_swiglu_backward(g, None, None, None, 256, None, None, 0, None) == ep.EP_OK


def test_grouped_matmul_refusals(lib):
    call = lambda g=groups(), x=rows8(), w=P, s=P, N=256, K=256, out=P: lib.ep_grouped_matmul(  # noqa: E731
        g, x, w, s, N, K, out, 0, None)
    for g in BAD_GROUPS:
        assert call(g=g) == BAD
    for x in BAD_ROWS:
        assert call(x=x) == BAD
    for kw in (dict(w=None), dict(w=P + 8), dict(s=None), dict(s=P + 2), dict(N=0), dict(N=4), dict(N=260),
               dict(K=0), dict(K=64), dict(K=200), dict(out=None), dict(out=P + 8), dict(N=1 << 30),
               dict(g=groups(rows=(1 << 31) - 1), N=1 << 20)):
        assert call(**kw) == BAD, kw


def test_grouped_matmul_swiglu_refusals(lib):
    call = lambda g=groups(), x=rows8(), w=P, s=P, F=256, K=256, rw=None, act=rows8(), pre=rows8(): (  # noqa: E731
        lib.ep_grouped_matmul_swiglu(g, x, w, s, F, K, rw, act, pre, 0, None))
    for g in BAD_GROUPS:
        assert call(g=g) == BAD
    for r in BAD_ROWS:
        assert call(x=r) == BAD and call(act=r) == BAD
        if r is not None:
            assert call(pre=r) == BAD
    for kw in (dict(w=None), dict(w=P + 8), dict(s=None), dict(F=0), dict(F=64), dict(F=192), dict(K=100),
               dict(rw=P + 2), dict(F=1 << 29)):
        assert call(**kw) == BAD, kw


def test_grouped_swiglu_backward_refusals(lib):
    call = lambda g=groups(), da=P, pre=rows8(), rw=None, F=256, out=rows8(), dw=None: (  # noqa: E731
        lib.ep_grouped_swiglu_backward(g, da, pre, rw, F, out, dw, 0, None))
    for g in BAD_GROUPS:
        assert call(g=g) == BAD
    for r in BAD_ROWS:
        assert call(pre=r) == BAD and call(out=r) == BAD
    for kw in (dict(da=None), dict(da=P + 8), dict(F=0), dict(F=130), dict(rw=P + 1), dict(dw=P + 2),
               dict(F=1 << 30)):
        assert call(**kw) == BAD, kw


def test_grouped_weight_grad_refusals(lib):
    call = lambda g=groups(), dy=rows8(), N=256, x=rows8(), K=256, dw=P: lib.ep_grouped_weight_grad(  # noqa: E731
        g, dy, N, x, K, dw, 0, None)
    for g in BAD_GROUPS:
        assert call(g=g) == BAD
    for r in BAD_ROWS:
        assert call(dy=r) == BAD and call(x=r) == BAD
    for kw in (dict(N=0), dict(N=64), dict(N=136), dict(K=0), dict(K=72), dict(dw=None), dict(dw=P + 8),
               dict(g=groups(num=4096), N=1 << 24, K=1 << 24)):
        assert call(**kw) == BAD, kw


def test_handle_calls_refuse_null(lib):
    assert lib.ep_em_get_groups(None, None, None, None) == BAD
    assert lib.ep_em_combine_weights(None, None, 0, None, None) == BAD
