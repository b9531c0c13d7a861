"""Infinities in mx4 operands: they are stored as 6 * 2^126, and products take
them for that number."""
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


def quantised(a):
    """(elements, scales, 64-bit values) of a."""
    e, s = ssg.mx4_quantize(a.cuda())
    return e, s, D.mx4_values(e.cpu().numpy(), s.cpu().numpy(), a.shape[1])


@pytest.mark.parametrize("N", [3, 300])
@pytest.mark.parametrize("side", ["activations", "weights"])
def test_products_of_stored_infinities(N, side):
    M, K = 70, 256
    X, W = D.randn((N, K), "f32", 1), D.randn((M, K), "f32", 2, 2.0 ** -8)
    big = X if side == "activations" else W
    big[1, 40], big[2, 0], big[2, 200] = float("inf"), float("-inf"), float("inf")
    if side == "weights":
        X *= 2.0 ** -8
    xe, xs, xv = quantised(X)
    we, ws, wv = quantised(W)
    v = xv if side == "activations" else wv
    assert v[1, 40] == 6 * 2.0 ** 126 and v[2, 0] == -6 * 2.0 ** 126
    back = ssg.mx4_dequantize(*((xe, xs) if side == "activations" else (we, ws)), K)
    assert back[1, 40] == float("inf") and back[2, 0] == float("-inf")
    D.check(ssg.mm_mx4(xe, we, ws, xscales=xs), xv @ wv.T, abs(xv) @ abs(wv).T, K, "mx4 x mx4")
    if side == "weights":
        Xh = X.bfloat16()
        xh = Xh.double().numpy()
        D.check(ssg.mm_mx4(Xh.cuda(), we, ws), xh @ wv.T, abs(xh) @ abs(wv).T, K, "16-bit x mx4")
