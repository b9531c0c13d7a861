"""Dense and grouped products at the ends of their operands: segments of one
row, memory of NaN around every operand, long contractions of few rows."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _mm as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    torch.cuda.init()
    return torch.device("cuda:0")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# every row its own segment, those of no expert included; one row more than a
# tile; tiles that begin 15 rows before their expert's first
@pytest.mark.parametrize("first,sizes,extra", [(1, [1] * 5, 1), (0, [1, 1], 0), (1, [0, 0, 1], 0), (0, [0] * 30 + [1], 1),
                                               (15, [17] * 6, 17), (15, [33, 0, 33, 33], 1), (15, [65, 129, 257], 2),
                                               (0, [0] * 70, 3)])
def test_small_segments(first, sizes, extra):
    E, N, M, K = len(sizes), first + sum(sizes) + extra, 72, 160
    offs = D.offsets(sizes, first)
    og = offs.cuda()
    X, W, dY = D.randn((N, K), "f16", 1), D.randn((E, M, K), "f16", 2, 0.1), D.randn((N, M), "f16", 3)
    e, s = D.random_mx4((E, M, K), 4)
    xe, xs = D.random_mx4((N, K), 5, 120, 130)
    x, w, d, w4 = X.double().numpy(), W.double().numpy(), dY.double().numpy(), D.mx4_values(e, s, K)
    f32 = dict(out_dtype=torch.float32)
    D.check(ssg.grouped_mm(X.cuda(), W.cuda(), og, **f32), *D.grouped(x, w, offs), K, "Y")
    D.check(ssg.grouped_mm_dx(dY.cuda(), W.cuda(), og, **f32), *D.grouped_dx(d, w, offs), M, "dX")
    D.check(ssg.grouped_mm_dw(dY.cuda(), X.cuda(), og, **f32), *D.grouped_dw(d, x, offs), N, "dW")
    D.check(ssg.grouped_mm_mx4(X.cuda(), dev(e), dev(s), og, **f32), *D.grouped(x, w4, offs), K, "mx4 weights")
    D.check(ssg.grouped_mm_mx4(dev(xe), dev(e), dev(s), og, xscales=dev(xs), **f32),
            *D.grouped(D.mx4_values(xe, xs, K), w4, offs), K, "mx4 x mx4")


def inside(t, before, after, poison):
    """t as a view of a larger tensor full of `poison`: `before` elements before
    each row, `after` behind it, and rows around the matrix."""
    big = torch.full((*t.shape[:-2], t.shape[-2] + 2, before + t.shape[-1] + after), poison, dtype=t.dtype).cuda()
    view = big[..., 1:-1, before:before + t.shape[-1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("before,after", [(0, 0), (1, 2), (2, 2), (4, 4), (8, 24), (3, 5)])
@pytest.mark.parametrize("M,K", [(264, 104), (390, 1058), (130, 999), (1024, 512)])
def test_nan_around_16_bit_operands(before, after, M, K):
    sizes = [300, 0, 17, 383]
    N, nan = sum(sizes), float("nan")
    offs = D.offsets(sizes)
    og = offs.cuda()
    X, W, dY = D.randn((N, K), "bf16", 7), D.randn((4, M, K), "bf16", 8, 0.1), D.randn((N, M), "bf16", 9)
    x, w, d = X.double().numpy(), W.double().numpy(), dY.double().numpy()
    Xv, Wv, Dv = (inside(t, before, after, nan) for t in (X, W, dY))
    D.check(ssg.grouped_mm(Xv, Wv, og), *D.grouped(x, w, offs), K, "Y")
    D.check(ssg.grouped_mm_dx(Dv, Wv, og), *D.grouped_dx(d, w, offs), M, "dX")
    D.check(ssg.grouped_mm_dw(Dv, Xv, og, out_dtype=torch.float32), *D.grouped_dw(d, x, offs), 383, "dW")


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("before,after", [(0, 0), (16, 32), (2, 2), (5, 6)])
@pytest.mark.parametrize("M,K,N", [(264, 416, 700), (300, 1058, 330), (1024, 608, 517)])
def test_nan_around_mx4_operands(x, before, after, M, K, N):
    """Elements around the matrices are 6, scales and 16-bit values NaN."""
    e, s = D.random_mx4((M, K), 31)
    wv = D.mx4_values(e, s, K)
    We, Ws = inside(dev(e), before, after, 0x77), inside(dev(s), before, after, 255)
    if x == "mx4":
        xe, xs = D.random_mx4((N, K), 32, 120, 130)
        xv = D.mx4_values(xe, xs, K)
        Y = ssg.mm_mx4(inside(dev(xe), before, after, 0x77), We, Ws, xscales=inside(dev(xs), before, after, 255))
    else:
        X = D.randn((N, K), x, 33)
        xv = X.double().numpy()
        Y = ssg.mm_mx4(inside(X, before, after, float("nan")), We, Ws)
    D.check(Y, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K, "mm_mx4")


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("M,K,N", [(48, 20001, 2), (16, 33024, 1), (200, 16384, 20), (130, 9000, 90)])
def test_long_contractions_of_few_rows(x, M, K, N):
    e, s = D.random_mx4((M, K), 41)
    wv = D.mx4_values(e, s, K)
    if x == "mx4":
        xe, xs = D.random_mx4((N, K), 42, 120, 130)
        xv = D.mx4_values(xe, xs, K)
        Y = ssg.mm_mx4(dev(xe), dev(e), dev(s), xscales=dev(xs))
    else:
        X = D.randn((N, K), x, 43)
        xv = X.double().numpy()
        Y = ssg.mm_mx4(X.cuda(), dev(e), dev(s))
    D.check(Y, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K, "mm_mx4")


@pytest.mark.parametrize("before,after", [(0, 0), (1, 0), (1, 1), (2, 1), (3, 4)])
@pytest.mark.parametrize("M,K,sizes", [(100, 257, [3, 0, 20]), (33, 1001, [1]), (520, 4097, [16, 17, 1]), (264, 640, [40])])
def test_few_rows_that_begin_anywhere(before, after, M, K, sizes):
    """16-bit rows at odd elements, with NaN around the operands."""
    offs, nan = D.offsets(sizes), float("nan")
    X, W = D.randn((sum(sizes), K), "f16", 51), D.randn((len(sizes), M, K), "f16", 52, 0.1)
    e, s = D.random_mx4((len(sizes), M, K), 53)
    Xv, x = inside(X, before, after, nan), X.double().numpy()
    D.check(ssg.grouped_mm(Xv, inside(W, before, after, nan), offs.cuda(), out_dtype=torch.float32),
            *D.grouped(x, W.double().numpy(), offs), K, "16-bit weights")
    D.check(ssg.grouped_mm_mx4(Xv, dev(e), dev(s), offs.cuda()), *D.grouped(x, D.mx4_values(e, s, K), offs), K,
            "mx4 weights")
