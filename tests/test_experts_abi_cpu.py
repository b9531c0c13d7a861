"""Routing, the order of expert rows, gather and combine on the CPU: what the entry
points refuse, on the host and before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from structured_sparse_gemm_amd import _abi
from tests import _experts as D

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails validation first
F16, BF16, I8, F32 = _abi.SSG_F16, _abi.SSG_BF16, _abi.SSG_I8, _abi.SSG_F32
NULL, SHAPE, STRIDE, DTYPE, WS, ALGO = (_abi.SSG_ERR_NULL, _abi.SSG_ERR_SHAPE, _abi.SSG_ERR_STRIDE,
                                        _abi.SSG_ERR_DTYPE, _abi.SSG_ERR_WORKSPACE, _abi.SSG_ERR_ALGO)


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def test_route_refusals(lib):
    def call(dt=F16, N=4, E=16, l=FAKE, ldl=16, bias=None, score=0, k=2, groups=1, top=1, gs=0, w=FAKE, ldw=2, e=FAKE,
             lde=2):
        return lib.ssg_route(dt, N, E, l, ldl, bias, score, k, groups, top, gs, 1, 1.0, w, ldw, e, lde, None)

    assert call(dt=I8) == DTYPE and call(score=2) == ALGO and call(gs=-1) == ALGO
    assert call(N=-1) == SHAPE and call(N=1 << 29) == SHAPE and call(N=1 << 28, E=64, ldl=64, k=16, ldw=16, lde=16) == SHAPE
    assert call(E=0) == SHAPE and call(E=1025, ldl=1025) == SHAPE
    assert call(k=0) == SHAPE and call(k=17) == SHAPE and call(E=256, ldl=256, k=65) == SHAPE
    assert call(groups=3) == SHAPE and call(groups=0) == SHAPE and call(groups=4, top=5) == SHAPE
    assert call(groups=4, top=0) == SHAPE and call(groups=8, top=1, k=3) == SHAPE
    assert call(E=130, ldl=130, groups=65) == SHAPE
    assert call(l=None) == NULL and call(w=None) == NULL and call(e=None) == NULL
    assert call(ldl=15) == STRIDE and call(ldw=1) == STRIDE and call(lde=1) == STRIDE
    assert call(N=0, l=None, w=None, e=None) == 0

    def back(dt=F16, N=4, E=16, dw=FAKE, lddw=2, l=FAKE, ldl=16, e=FAKE, lde=2, score=0, k=2, d=FAKE, ldd=16):
        return lib.ssg_route_backward(dt, N, E, dw, lddw, l, ldl, e, lde, score, k, 1, 1.0, d, ldd, None)

    assert back(dt=I8) == DTYPE and back(score=9) == ALGO and back(k=0) == SHAPE and back(E=0) == SHAPE
    assert back(dw=None) == NULL and back(l=None) == NULL and back(e=None) == NULL and back(d=None) == NULL
    assert back(lddw=1) == STRIDE and back(ldl=15) == STRIDE and back(lde=1) == STRIDE and back(ldd=15) == STRIDE
    assert back(N=0, dw=None, l=None, e=None, d=None) == 0


def test_order_refusals(lib):
    def call(N=4, k=2, E=8, e=FAKE, lde=2, offs=FAKE, rows=FAKE, pos=FAKE, ws=None, size=0):
        return lib.ssg_expert_order(N, k, E, e, lde, offs, rows, pos, ws, size, None)

    assert call(N=-1) == SHAPE and call(k=-1) == SHAPE and call(k=65, lde=65) == SHAPE
    assert call(E=-1) == SHAPE and call(E=1025) == SHAPE and call(N=1 << 28, k=8, lde=8) == SHAPE
    assert call(e=None) == NULL and call(offs=None) == NULL and call(rows=None) == NULL and call(pos=None) == NULL
    assert call(lde=1) == STRIDE
    f = lib.ssg_expert_order_workspace_bytes
    assert f(4096, 1, 64) == 0 and f(-1, 2, 8) == 0 and f(4, 2, 2000) == 0
    need = f(4097, 1, 64)
    assert need == 5 * 64 * 4
    big = dict(N=4097, k=1, E=64, lde=1)
    assert call(**big) == WS and call(**big, ws=FAKE, size=need - 1) == WS
    assert call(**big, ws=ctypes.c_void_p(0x1002), size=need) == WS
    assert call(**big, size=_abi.SSG_WS_ASK) == WS
    assert f(1 << 25, 8, 1024) <= 256 * 1024 * 4


def test_rows_refusals(lib):
    def gather(dt=F16, N=4, k=2, C=8, X=FAKE, ldx=8, pos=FAKE, rows=FAKE, Y=FAKE, ldy=8):
        return lib.ssg_expert_gather(dt, N, k, C, X, ldx, pos, rows, Y, ldy, None)

    def combine(dt=F16, out=F16, N=4, k=2, C=8, Y=FAKE, ldy=8, pos=FAKE, w=FAKE, ldw=2, O=FAKE, ldo=8):
        return lib.ssg_expert_combine(dt, out, N, k, C, Y, ldy, pos, w, ldw, O, ldo, None)

    def back(dt=F16, N=4, k=2, C=8, dO=FAKE, lddo=8, Y=FAKE, ldy=8, pos=FAKE, rows=FAKE, w=FAKE, ldw=2, dY=FAKE, lddy=8,
             dw=FAKE, lddw=2):
        return lib.ssg_expert_combine_backward(dt, N, k, C, dO, lddo, Y, ldy, pos, rows, w, ldw, dY, lddy, dw, lddw, None)

    for f in (gather, combine, back):
        assert f(dt=I8) == DTYPE and f(N=-1) == SHAPE and f(k=65) == SHAPE and f(C=-1) == SHAPE and f(C=1 << 29) == SHAPE
        assert f(N=1 << 28, k=8) == SHAPE and f(pos=None) == NULL and f(ldy=7) == STRIDE and f(Y=None) == NULL
    assert gather(X=None) == NULL and gather(rows=None) == NULL and gather(ldx=7) == STRIDE
    assert combine(out=BF16) == DTYPE and combine(dt=F32, out=F16) == DTYPE and combine(O=None) == NULL
    assert combine(ldw=1) == STRIDE and combine(ldo=7) == STRIDE
    assert back(dO=None) == NULL and back(w=None) == NULL and back(dY=None) == NULL and back(dw=None) == NULL
    assert back(rows=None) == NULL and back(lddo=7) == STRIDE and back(lddy=7) == STRIDE and back(lddw=1) == STRIDE
    assert gather(N=0, X=None, pos=None, rows=None, Y=None) == 0
    assert combine(N=0, Y=None, pos=None, w=None, O=None) == 0
    assert back(N=0, dO=None, Y=None, pos=None, rows=None, w=None, dY=None, dw=None) == 0


def test_python_refusals():
    l, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    w, rows = torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32)
    Y = torch.zeros(8, 6)

    def status(f, *a, **k):
        with pytest.raises(ssg.SsgError) as err:
            f(*a, **k)
        return err.value.status

    assert status(ssg.route, l, 2) == NULL                        # not on a device
    assert status(ssg.route, l[0], 2) == SHAPE
    assert status(ssg.route, l.double(), 2) == DTYPE
    assert status(ssg.route, l.t(), 2) == STRIDE
    assert status(ssg.route_backward, w, l, e) == NULL
    assert status(ssg.expert_order, e, 8) == NULL
    assert status(ssg.expert_order, e.long(), 8) == DTYPE
    assert status(ssg.expert_order, e[0], 8) == SHAPE
    assert status(ssg.expert_gather, torch.zeros(4, 6), e, rows) == NULL
    assert status(ssg.expert_combine, Y, e, w) == NULL
    assert status(ssg.expert_combine_backward, torch.zeros(4, 6), Y, e, rows, w) == NULL


def test_definitions():
    """The definitions against a few results worked out by hand."""
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    w, e = D.route(l, 2)
    assert e.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    w, e = D.route(l, 2, renorm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    w, e = D.route(l, 2, groups=2, top_groups=1, group_score="top2")
    assert e.tolist() == [[2, 3]]
    w, e = D.route(l, 1, bias=np.array([0.9, 0.0, 0.0, 0.0]))
    assert e.tolist() == [[0]] and w[0, 0] == 1.0
    offs, rows, pos = D.order(np.array([[1, 0], [-1, 1]]), 3)
    assert offs.tolist() == [0, 1, 3, 3] and rows.tolist() == [1, 0, 3, -1] and pos.tolist() == [[1, 0], [-1, 2]]
    g, _ = D.route_grad(np.array([[1.0, 0.0]]), l, np.array([[2, 1]]))
    assert np.allclose(g, [[0, -2 / 9, 2 / 9, 0]])
