"""mx4 weights with blocks of zeros against 16-bit activations: such blocks are
exact under every scale, and have no part in how the others are multiplied."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _mm as D

pytestmark = pytest.mark.gpu

# (M, K, N) for the few-token kernels, with and without shared scales, and the tiled ones
SHAPES = [(200, 1056, 1), (70, 96, 20), (520, 4128, 3), (11008, 512, 16), (16, 20000, 2), (300, 416, 300), (1024, 1000, 600)]


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    torch.cuda.init()
    return torch.device("cuda:0")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def zero_blocks(M, K, seed):
    """Random mx4 rows in which some blocks, and all of some rows, hold +0 and -0."""
    e, s = D.random_mx4((M, K), seed)
    g = np.random.default_rng(seed + 1)
    zero = g.random(s.shape) < 0.05
    zero[[3, M // 2, M - 1]] = True
    signs = g.choice(np.array([0x00, 0x08, 0x80, 0x88], dtype=np.uint8), e.shape)
    return np.where(np.repeat(zero, 16, axis=1), signs, e), s, zero


def product(grouped, X, e, s):
    if not grouped:
        return ssg.mm_mx4(X, dev(e), dev(s))
    n = X.shape[0]
    offs = torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32).cuda()
    return ssg.grouped_mm_mx4(X, *(dev(t[None]).expand(3, *t.shape) for t in (e, s)), offs)


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_scales_of_zero_blocks_do_not_matter(x, grouped, M, K, N):
    e, s, zero = zero_blocks(M, K, 3)
    X = D.randn((N, K), x, 4)
    xv, wv = X.double().numpy(), D.mx4_values(e, s, K)
    want = product(grouped, X.cuda(), e, np.where(zero, 120, s).astype(np.uint8))
    D.check(want, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K, "zero blocks")
    anything = np.random.default_rng(5).integers(0, 255, s.shape).astype(np.uint8)
    for scales in (np.zeros_like(s), np.full_like(s, 254), anything):
        got = product(grouped, X.cuda(), e, np.where(zero, scales, s).astype(np.uint8))
        assert torch.equal(got, want)


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_scales_that_matter_beside_zero_blocks(x, M, K, N):
    # one element of 0.5 in the last row's last block, under a scale past the
    # 16-bit types; and a NaN scale over zeros
    e, s, zero = zero_blocks(M, K, 6)
    s = np.where(zero, 0, s).astype(np.uint8)
    e[M - 1, -16], s[M - 1, -1] = 0x01, 200
    X = D.randn((N, K), x, 7)
    xv, wv = X.double().numpy(), D.mx4_values(e, s, K)
    Y = ssg.mm_mx4(X.cuda(), dev(e), dev(s))
    D.check(Y, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K, "scale 200")
    s[3, 1] = 255
    Y = ssg.mm_mx4(X.cuda(), dev(e), dev(s)).cpu()
    assert torch.isnan(Y[:, 3]).all()
    assert torch.isfinite(Y[:, :3]).all() and torch.isfinite(Y[:, 4:]).all()


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("N", [1, 16, 300])
def test_quantised_rows_of_zeros(x, N):
    W = D.randn((264, 4096), "bf16", 8, 0.02)
    W[::7] = 0
    e, s = ssg.mx4_quantize(W.cuda())
    assert (s[::7] == 0).all()
    X = D.randn((N, 4096), x, 9).cuda()
    Y = ssg.mm_mx4(X, e, s)
    other = torch.where(s == 0, torch.full_like(s, 120), s)
    assert (Y[:, ::7] == 0).all() and torch.equal(Y, ssg.mm_mx4(X, e, other))
