"""The mx4 and expert-grouped entry points on the CPU: what they refuse, on the
host and before anything is enqueued, and the workspace they ask for."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from structured_sparse_gemm_amd import _abi
from tests import _mm as D

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails validation first
F16, BF16, I8, F32, MX4 = _abi.SSG_F16, _abi.SSG_BF16, _abi.SSG_I8, _abi.SSG_F32, _abi.SSG_MX4
NULL, SHAPE, STRIDE, DTYPE, FORMAT, WS = (_abi.SSG_ERR_NULL, _abi.SSG_ERR_SHAPE, _abi.SSG_ERR_STRIDE,
                                          _abi.SSG_ERR_DTYPE, _abi.SSG_ERR_FORMAT, _abi.SSG_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def test_definitions_agree():
    # the definition's quantiser round-trips every code at every scale, and its
    # nearest-code search agrees with a search over the eight values in 64 bits
    e, s = D.random_mx4((6, 96), 1, 10, 240)
    v = D.mx4_values(e, s, 96)
    e2, s2 = D.mx4_quantize(v)
    assert np.array_equal(D.mx4_values(e2, s2, 96), v)
    a = np.random.default_rng(2).standard_normal((8, 64))
    e, s = D.mx4_quantize(a)
    scale = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1)
    q = np.minimum(np.abs(a) / scale, 6.0)
    nearest = np.abs(q[:, :, None] - D.CODES).min(axis=2)
    assert np.array_equal(np.abs(np.abs(D.mx4_values(e, s, 64)) / scale - q), nearest)


def test_columns(lib):
    for K, nb in [(0, 0), (1, 1), (32, 1), (33, 2), (4096, 128)]:
        assert lib.ssg_mx4_elem_cols(K) == 16 * nb == ssg.ssg_mx4_elem_cols(K)
        assert lib.ssg_mx4_scale_cols(K) == nb == ssg.ssg_mx4_scale_cols(K)


def test_quantize_refusals(lib):
    for f in (lib.ssg_mx4_quantize, ):
        assert f(I8, 4, 64, FAKE, 64, FAKE, 32, FAKE, 2, None) == DTYPE
        assert f(F16, -1, 64, FAKE, 64, FAKE, 32, FAKE, 2, None) == SHAPE
        assert f(F16, 4, 64, None, 64, FAKE, 32, FAKE, 2, None) == NULL
        assert f(F16, 4, 64, FAKE, 63, FAKE, 32, FAKE, 2, None) == STRIDE
        assert f(F16, 4, 64, FAKE, 64, FAKE, 31, FAKE, 2, None) == STRIDE
        assert f(F16, 4, 65, FAKE, 65, FAKE, 48, FAKE, 2, None) == STRIDE
        assert f(F16, 0, 64, None, 64, None, 32, None, 2, None) == 0
    assert lib.ssg_mx4_dequantize(I8, 4, 64, FAKE, 32, FAKE, 2, FAKE, 64, None) == DTYPE
    assert lib.ssg_mx4_dequantize(F32, 4, 64, FAKE, 32, None, 2, FAKE, 64, None) == NULL
    assert lib.ssg_mx4_dequantize(F32, 4, 64, FAKE, 32, FAKE, 2, FAKE, 60, None) == STRIDE


def test_mm_mx4_refusals(lib):
    f = lib.ssg_mm_mx4

    def call(x=BF16, y=F32, M=8, N=4, K=64, X=FAKE, ldx=64, xs=None, ldxs=0, W=FAKE, ldw=32, S=FAKE, lds=2, Y=FAKE,
             ldy=8):
        return f(x, y, M, N, K, X, ldx, xs, ldxs, W, ldw, S, lds, Y, ldy, None, 0, None)

    assert call(x=I8) == DTYPE and call(x=F32) == DTYPE
    assert call(y=F16) == DTYPE and call(x=F16, y=BF16) == DTYPE and call(y=I8) == DTYPE
    assert call(M=-1) == SHAPE and call(N=1 << 31) == SHAPE and call(K=-64) == SHAPE
    assert call(X=None) == NULL and call(W=None) == NULL and call(S=None) == NULL and call(Y=None) == NULL
    assert call(ldx=63) == STRIDE and call(ldw=31) == STRIDE and call(lds=1) == STRIDE and call(ldy=7) == STRIDE
    assert call(ldx=1 << 22) == STRIDE
    assert call(xs=FAKE, ldxs=2) == FORMAT                       # scales for 16-bit activations
    assert call(x=MX4, ldx=32) == NULL                           # and none for mx4 ones
    assert call(x=MX4, ldx=31, xs=FAKE, ldxs=2) == STRIDE
    assert call(x=MX4, ldx=32, xs=FAKE, ldxs=1) == STRIDE
    assert call(N=0, X=None, Y=None) == 0 and call(M=0, W=None, S=None, Y=None) == 0


def test_grouped_refusals(lib):
    def fwd(x=F16, y=F16, E=2, M=8, N=4, K=16, X=FAKE, ldx=16, W=FAKE, ldw=16, st=128, offs=FAKE, Y=FAKE, ldy=8):
        return lib.ssg_grouped_mm(x, y, E, M, N, K, X, ldx, W, ldw, st, offs, Y, ldy, None, 0, None)

    def dx(x=F16, y=F16, E=2, M=8, N=4, K=16, dY=FAKE, lddy=8, W=FAKE, ldw=16, st=128, offs=FAKE, Y=FAKE, ldy=16):
        return lib.ssg_grouped_mm_dx(x, y, E, M, N, K, dY, lddy, W, ldw, st, offs, Y, ldy, None, 0, None)

    def dw(x=F16, y=F16, E=2, M=8, N=4, K=16, dY=FAKE, lddy=8, X=FAKE, ldx=16, offs=FAKE, W=FAKE, ldw=16, st=128):
        return lib.ssg_grouped_mm_dw(x, y, E, M, N, K, dY, lddy, X, ldx, offs, W, ldw, st, None, 0, None)

    for f in (fwd, dx, dw):
        assert f(x=MX4) == DTYPE and f(x=I8) == DTYPE and f(y=BF16) == DTYPE
        assert f(E=-1) == SHAPE and f(N=-1) == SHAPE and f(E=1 << 20) == SHAPE
        assert f(offs=None) == NULL and f(W=None) == NULL
        assert f(ldw=15) == STRIDE
    assert fwd(X=None) == NULL and dx(dY=None) == NULL and dw(dY=None) == NULL and dw(X=None) == NULL
    assert fwd(ldx=15) == STRIDE and dx(lddy=7) == STRIDE and dw(ldx=15) == STRIDE and dx(ldy=15) == STRIDE
    assert fwd(N=0, X=None, Y=None) == 0 and dx(N=0, dY=None, Y=None) == 0 and dw(E=0, W=None) == 0

    def mx4(x=F16, y=F16, E=2, M=8, N=4, K=64, X=FAKE, ldx=64, xs=None, ldxs=0, W=FAKE, ldw=32, st=256, S=FAKE, lds=2,
            sts=16, offs=FAKE, Y=FAKE, ldy=8):
        return lib.ssg_grouped_mm_mx4(x, y, E, M, N, K, X, ldx, xs, ldxs, W, ldw, st, S, lds, sts, offs, Y, ldy, None,
                                      0, None)

    assert mx4(x=I8) == DTYPE and mx4(y=BF16) == DTYPE and mx4(offs=None) == NULL and mx4(S=None) == NULL
    assert mx4(lds=1) == STRIDE and mx4(xs=FAKE) == FORMAT and mx4(x=MX4, ldx=32) == NULL


def test_workspace(lib):
    A16, A2 = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)
    f = lib.ssg_grouped_mm_workspace_bytes
    # few rows: nothing; many: nothing where the rows are aligned and the chip is full
    assert f(F16, 8, 4096, 2, 4096, A16, 4096, A16, 4096, 4096 * 4096, FAKE) == 0
    assert f(F16, 8, 4096, 8192, 4096, A16, 4096, A16, 4096, 4096 * 4096, FAKE) == 0
    # an operand off 16-byte alignment is copied to rows of a multiple of 16 bytes
    need = f(F16, 8, 4096, 8192, 4096, A2, 4096, A16, 4096, 4096 * 4096, FAKE)
    assert need == 8192 * 4096 * 2
    need = f(F16, 8, 4096, 8192, 4001, A16, 4001, A16, 4001, 4096 * 4001, FAKE)
    assert need == 8192 * 4008 * 2 + 8 * 4096 * 4008 * 2
    # refused arguments need none, and a product without its workspace enqueues nothing
    assert f(I8, 8, 4096, 8192, 4001, A16, 4001, A16, 4001, 4096 * 4001, FAKE) == 0
    g = lib.ssg_grouped_mm
    args = (F16, F16, 8, 4096, 8192, 4001, A16, 4001, A16, 4001, 4096 * 4001, FAKE, FAKE, 4096)
    assert g(*args, None, 0, None) == WS and g(*args, FAKE, need - 1, None) == WS
    assert g(*args, ctypes.c_void_p(0x1008), need, None) == WS
    assert "workspace" in lib.ssg_last_error().decode()


def test_python_refusals():
    h = torch.zeros(4, 64, dtype=torch.float16)
    u, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    w, offs = torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)

    def status(f, *a, **k):
        with pytest.raises(ssg.SsgError) as e:
            f(*a, **k)
        return e.value.status

    assert status(ssg.mx4_quantize, h) == NULL                   # not on a device
    assert status(ssg.mx4_quantize, h.to(torch.int8)) == DTYPE
    assert status(ssg.mx4_quantize, h[0]) == SHAPE
    assert status(ssg.mm_mx4, h, u, s) == NULL
    assert status(ssg.mm_mx4, h, u.to(torch.int8), s) == DTYPE
    assert status(ssg.mm_mx4, h[:, :32], u, s) == SHAPE
    assert status(ssg.mm_mx4, h, u, s[:, :1]) == SHAPE
    assert status(ssg.mm_mx4, h.float(), u, s) == DTYPE
    assert status(ssg.mm_mx4, u, u, s, xscales=s[:4]) == SHAPE
    assert status(ssg.grouped_mm_mx4, h, u, s, offs) == SHAPE
    assert status(ssg.grouped_mm, h, w, offs) == NULL
    assert status(ssg.grouped_mm, h, w.bfloat16(), offs) == DTYPE
    assert status(ssg.grouped_mm, h[:, :60], w, offs) == SHAPE
    assert status(ssg.grouped_mm, h, w[0], offs) == SHAPE
    assert status(ssg.grouped_mm_dx, h, w, offs) == SHAPE
    assert status(ssg.grouped_mm_dw, h, h[:3], offs) == SHAPE


def test_compiled_calls_take_only_device_tensors():
    # built beside the library; anything it does not take is left to the
    # Python binding, which says what is wrong
    calls = _abi.torch_calls()
    assert calls is not None
    h, u, s = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    w, offs = torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    assert calls.mx4_quantize(h) is None and calls.mx4_quantize(None) is None and calls.mx4_quantize(h, h) is None
    assert calls.mx4_dequantize(u, s, 64, torch.float16) is None
    assert calls.mx4_dequantize(u, s, "64", torch.float16) is None and calls.mx4_dequantize(u, s, 64, 1) is None
    assert calls.mx4_product(h, None, u, s, None, torch.float32) is None
    assert calls.mx4_product(h, None, u, s, offs, 3) is None and calls.mx4_product(1, 2, 3) is None
    for kind in (0, 1, 2):
        assert calls.grouped_product(kind, h, w, offs, torch.float16) is None
        assert calls.grouped_product(kind, "x", w, offs, torch.float16) is None
