"""NaN of every payload stays NaN in 8 bits, and in the products of its row alone."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _fp8 as D

pytestmark = pytest.mark.gpu

# quiet ones (the last 32 payloads among them), signalling ones, of both signs
BITS = [0x7FC00000, 0x7FC00001, 0x7FFFFFDF, 0x7FFFFFE0, 0x7FFFFFE1, 0x7FFFFFFF, 0xFFC00000, 0xFFFFFFE0, 0xFFFFFFFF,
        0x7F800001, 0x7FBFFFFF, 0xFF800001, 0xFFBFFFFF]


def nans(R, K, at, scale=1.0):
    """fp32 [R, K] with NaN number i at row i, column at + i."""
    a = (D.randn((R, K), "f32", R + K) * scale).numpy().view(np.uint32)
    for i, b in enumerate(BITS):
        a[i, at + i] = b
    return torch.from_numpy(a.view(np.float32))


@pytest.mark.parametrize("scale", [1.0, 1e-30])              # (and blocks whose scale is far below 1)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize(block, transpose, scale):
    a = nans(40, 300, 120, scale)
    e, s = ssg.fp8_quantize((a.t().contiguous() if transpose else a).cuda(), block=block, transpose=transpose)
    got = D.codes_of(e)
    codes, scales = D.quantize(a.double().numpy(), block)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scales)
    assert ((got[torch.isnan(a).numpy()] & 0x7F) == 0x7F).all()
    rest = ~torch.isnan(a).numpy()
    assert np.array_equal(got[rest], codes[rest])
    back = ssg.fp8_dequantize(e, s)
    assert torch.equal(torch.isnan(back.cpu()), torch.isnan(a))


@pytest.mark.parametrize("N", [13, 700])                      # few and many rows
def test_products_of_fp32_activations(N):
    M, K = 150, 300
    X = nans(N, K, 0)
    w, ws = ssg.fp8_quantize(D.randn((M, K), "bf16", 2).cuda(), block=128)
    Y = ssg.mm_fp8(X.cuda(), w, ws)
    assert torch.isnan(Y[:len(BITS)]).all()
    assert torch.isfinite(Y[len(BITS):]).all()
    offs = torch.tensor([0, N], dtype=torch.int32).cuda()
    Z = ssg.grouped_mm_fp8(X.cuda(), w[None], ws[None], offs)
    assert torch.equal(torch.isnan(Z), torch.isnan(Y))


# a signalling NaN of each type: behind the largest number of its eight, before it, alone
SIGNALLING = {"f32": 0x7F800001, "bf16": 0x7F81, "f16": 0x7D01}


def signalling(R, K, dt):
    a = D.randn((R, K), dt, R + K) * 0.01
    bits = a.view(torch.int32 if dt == "f32" else torch.int16)
    for r in range(0, R, 2):
        at = 8 * (r % 30)
        a[r, at] = 3.0                                        # the largest of row r
        bits[r, at + 1 + r % 7] = SIGNALLING[dt]
        bits[r, (at + 8) % K] = SIGNALLING[dt]
        if r % 4:
            bits[r, at - 1] = SIGNALLING[dt]
    return a


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
def test_signalling_ones_do_not_count_for_the_scale(transpose, block, dt):
    a = signalling(60, 300, dt)
    e, s = ssg.fp8_quantize((a.t().contiguous() if transpose else a).cuda(), block=block, transpose=transpose)
    codes, scales = D.quantize(a.double().numpy(), block)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scales)
    got, nan = D.codes_of(e), torch.isnan(a).numpy()
    assert ((got[nan] & 0x7F) == 0x7F).all() and np.array_equal(got[~nan], codes[~nan])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [13, 700])
def test_activations_with_signalling_ones(N, dt):
    X = signalling(N, 300, dt).cuda()
    w, ws = ssg.fp8_quantize(D.randn((150, 300), "bf16", 2).cuda(), block=128)
    x, xs = ssg.fp8_quantize(X)
    Y = ssg.mm_fp8(X, w, ws)
    assert torch.isnan(Y[::2]).all() and torch.isfinite(Y[1::2]).all()
    # rounded in the call as before it: other rows, and the scales of these, are the same
    assert torch.equal(Y[1::2], ssg.mm_fp8(x, w, ws, xscales=xs)[1::2])
    clean = torch.where(torch.isnan(X), torch.zeros_like(X), X)
    assert torch.equal(ssg.fp8_quantize(clean)[1], xs)
