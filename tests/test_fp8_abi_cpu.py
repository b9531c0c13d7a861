"""8-bit floats with a scale for each block of 128 on the CPU: what the entry points
refuse, on the host and before anything is enqueued, and the workspace they ask for."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from structured_sparse_gemm_amd import _abi
from tests import _fp8 as D

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails validation first
F16, BF16, I8, F32, I32, E4M3, E5M2 = (_abi.SSG_F16, _abi.SSG_BF16, _abi.SSG_I8, _abi.SSG_F32, _abi.SSG_I32,
                                       _abi.SSG_E4M3, _abi.SSG_E5M2)
NULL, SHAPE, STRIDE, DTYPE, FORMAT, WS = (_abi.SSG_ERR_NULL, _abi.SSG_ERR_SHAPE, _abi.SSG_ERR_STRIDE,
                                          _abi.SSG_ERR_DTYPE, _abi.SSG_ERR_FORMAT, _abi.SSG_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def test_definitions():
    b = torch.arange(256, dtype=torch.uint8)
    v = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(D.values(b.numpy()[None], np.ones((1, 2)))[0], v, equal_nan=True)
    assert np.array_equal(D.nearest(v) & 0x7F, b.numpy() & 0x7F)
    q = np.random.default_rng(1).uniform(-448, 448, 5000) * np.exp2(np.random.default_rng(2).integers(-16, 1, 5000))
    near = np.abs(np.abs(q)[:, None] - D.CODES).min(axis=1)
    assert np.array_equal(np.abs(np.abs(q) - D.CODES[D.nearest(q) & 0x7F]), near)


def test_quantize_refusals(lib):
    def call(dt=F16, B=1, R=4, K=200, A=FAKE, lda=200, block=1, tr=0, e=FAKE, lde=200, stride=800, s=FAKE, row=2, blk=1,
             mat=8):
        return lib.ssg_fp8_quantize(dt, B, R, K, A, lda, 0, block, tr, e, lde, stride, s, row, blk, mat, None)

    assert call(dt=I8) == DTYPE and call(dt=E4M3) == DTYPE and call(block=64) == FORMAT and call(block=0) == FORMAT
    assert call(B=-1) == SHAPE and call(R=-1) == SHAPE and call(K=-1) == SHAPE and call(R=1 << 29) == SHAPE
    assert call(K=1 << 29, lda=1 << 29, lde=1 << 29) == SHAPE and call(B=1 << 20) == SHAPE
    assert call(A=None) == NULL and call(e=None) == NULL and call(s=None) == NULL
    assert call(lda=199) == STRIDE and call(lde=199) == STRIDE and call(row=-1) == STRIDE
    assert call(row=0) == STRIDE and call(blk=0) == STRIDE and call(row=1, blk=1) == STRIDE   # scales that share a place
    assert call(row=1, blk=3) == STRIDE and call(row=1 << 29) == STRIDE
    # matrices of a stack that share a place, or interleave in a way that may
    assert call(B=3, stride=0) == STRIDE and call(B=3, stride=799) == STRIDE and call(B=3, stride=200) == STRIDE
    assert call(B=3, mat=0) == STRIDE and call(B=3, mat=7) == STRIDE and call(B=3, stride=1 << 62) == STRIDE
    assert call(B=3, lde=599, stride=200) == STRIDE
    assert call(tr=1, lde=3) == STRIDE and call(tr=1, lde=200, row=0) == STRIDE
    assert call(R=1 << 28, K=1 << 20, lda=1 << 20, lde=1 << 20, row=1 << 13) == SHAPE
    assert call(R=0, A=None, e=None, s=None) == 0 and call(K=0, A=None, e=None, s=None, lda=0, lde=0) == 0

    def back(dt=F16, B=1, R=4, K=200, e=FAKE, lde=200, block=1, s=FAKE, row=2, blk=1, d=FAKE, ldd=200, stride=800):
        return lib.ssg_fp8_dequantize(dt, B, R, K, e, lde, 0, block, s, row, blk, 0, d, ldd, stride, None)

    assert back(dt=I8) == DTYPE and back(block=2) == FORMAT and back(R=-1) == SHAPE
    assert back(e=None) == NULL and back(s=None) == NULL and back(d=None) == NULL
    assert back(lde=199) == STRIDE and back(ldd=199) == STRIDE and back(blk=-1) == STRIDE
    assert back(B=2, stride=0) == STRIDE and back(B=2, stride=799) == STRIDE and back(B=2, stride=200) == STRIDE


def test_product_refusals(lib):
    def mm(x=BF16, y=F32, M=8, N=4, K=200, X=FAKE, ldx=200, xs=None, xsr=0, xsk=0, W=FAKE, ldw=200, wb=128, S=FAKE, sr=2,
           sk=1, Y=FAKE, ldy=8):
        return lib.ssg_mm_fp8(x, y, M, N, K, X, ldx, xs, xsr, xsk, W, ldw, wb, S, sr, sk, Y, ldy, None, 0, None)

    def grouped(x=BF16, y=F32, E=2, M=8, N=4, K=200, X=FAKE, ldx=200, xs=None, xsr=0, xsk=0, W=FAKE, ldw=200, wb=128,
                S=FAKE, sr=2, sk=1, Y=FAKE, ldy=8, offs=FAKE):
        return lib.ssg_grouped_mm_fp8(x, y, E, M, N, K, X, ldx, xs, xsr, xsk, W, ldw, 1600, wb, S, sr, sk, 2, offs, Y, ldy,
                                      None, 0, None)

    for f in (mm, grouped):
        assert f(x=I8) == DTYPE and f(x=E5M2) == DTYPE and f(y=I32) == DTYPE and f(y=E4M3) == DTYPE
        assert f(wb=32) == FORMAT and f(xs=FAKE) == FORMAT
        assert f(M=-1) == SHAPE and f(N=1 << 29) == SHAPE and f(K=1 << 29) == SHAPE
        assert f(X=None) == NULL and f(W=None) == NULL and f(S=None) == NULL and f(Y=None) == NULL
        assert f(x=E4M3) == NULL                                 # and no scales for e4m3 ones
        assert f(ldx=199) == STRIDE and f(ldw=199) == STRIDE and f(ldy=7) == STRIDE
        assert f(ldx=1 << 21) == STRIDE and f(ldw=1 << 22) == STRIDE and f(x=F32, ldx=1 << 20) == STRIDE
        assert f(sr=-1) == STRIDE and f(sk=1 << 29) == STRIDE and f(x=E4M3, xs=FAKE, xsr=-1) == STRIDE
        assert f(N=0, X=None, Y=None) == 0 and f(M=0, W=None, S=None, Y=None) == 0
    assert grouped(E=-1) == SHAPE and grouped(E=1 << 20) == SHAPE and grouped(offs=None) == NULL


def test_workspace(lib):
    f = lib.ssg_mm_fp8_workspace_bytes
    args = (4096, FAKE, 4096, None, 0, 0, FAKE, 4096, 128, FAKE, 32, 1)
    f = lambda x, *a, f=f: f(x, BF16, *a)                         # noqa: E731
    assert f(BF16, 4096, 1, *args) == 0                          # few rows are rounded on the way
    need = f(BF16, 4096, 2048, *args)
    assert need >= 2048 * 4096 + 2048 * 32 * 4                   # many in a pass of their own
    assert f(E4M3, 4096, 2048, 4096, FAKE, 4096, FAKE, 1, 2048, FAKE, 4096, 128, FAKE, 32, 1) == 0
    # elements off 4 bytes and scales by rows are copied
    odd = ctypes.c_void_p(0x1001)
    assert f(E4M3, 4096, 2048, 4096, odd, 4096, FAKE, 1, 2048, FAKE, 4096, 128, FAKE, 32, 1) == 2048 * 4096
    assert f(E4M3, 4096, 2048, 4096, FAKE, 4096, FAKE, 32, 1, FAKE, 4096, 128, FAKE, 32, 1) == 2048 * 32 * 4
    assert f(I8, 4096, 2048, *args) == 0
    g = lib.ssg_mm_fp8
    call = (BF16, BF16, 4096, 2048, *args, FAKE, 4096)
    assert g(*call, None, 0, None) == WS and g(*call, FAKE, need - 1, None) == WS
    assert g(*call, ctypes.c_void_p(0x1008), need, None) == WS
    assert g(*call, None, _abi.SSG_WS_ASK, None) == WS


def test_python_refusals():
    f = torch.float8_e4m3fn
    h, w = torch.zeros(4, 200, dtype=torch.float16), torch.zeros(8, 200).to(f)
    s, w3 = torch.zeros(1, 2), torch.zeros(2, 8, 200).to(f)
    offs = torch.zeros(3, dtype=torch.int32)

    def status(fn, *a, **k):
        with pytest.raises(ssg.SsgError) as e:
            fn(*a, **k)
        return e.value.status

    assert status(ssg.fp8_quantize, h) == NULL                   # not on a device
    assert status(ssg.fp8_quantize, h.to(torch.int8)) == DTYPE
    assert status(ssg.fp8_quantize, h[0]) == SHAPE and status(ssg.fp8_quantize, h, block=64) == FORMAT
    assert status(ssg.fp8_dequantize, w, s) == NULL
    assert status(ssg.fp8_dequantize, h, s) == DTYPE
    assert status(ssg.mm_fp8, h, w, s) == NULL
    assert status(ssg.mm_fp8, h, w.to(torch.float8_e5m2), s) == DTYPE
    assert status(ssg.mm_fp8, h[:, :100], w, s) == SHAPE
    assert status(ssg.mm_fp8, w, w, s) == FORMAT                 # e4m3 without scales
    assert status(ssg.grouped_mm_fp8, h, w, s, offs) == SHAPE
    assert status(ssg.grouped_mm_fp8, h, w3, s, offs) in (SHAPE, NULL)
