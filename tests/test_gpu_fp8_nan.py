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
