"""Products of operands past 32-bit offsets, and of many experts.  The operands
are outer products of small whole numbers, so that every sum is exact."""
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
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def cycle(n, period, low):
    """low, low + 1, .., for `period` numbers, and again."""
    return (torch.arange(n, device="cuda") % period + low).float()


def outer(a, b, dt=torch.bfloat16):
    return a.to(dt)[:, None] * b.to(dt)[None, :]


# rows of whole 16-byte pieces, and rows that end inside one (the gradients copy them)
@pytest.mark.parametrize("K", [2048, 1026])
def test_tokens_past_32_bits(K):
    N, M = (1 << 32) // (2 * K) + 40_000, 70
    assert N * K * 2 > 1 << 32
    a, b = cycle(N, 7, -3), cycle(K, 5, -2)
    c, d = cycle(N, 3, -1), cycle(M, 4, -1)
    X, dY = outer(a, b), outer(c, d)
    W = torch.stack([outer(cycle(M, 3, -1) * s, cycle(K, 3, 0)) for s in (1.0, 2.0)])
    cut = N - 30_000
    offs = torch.tensor([17, cut, N - 5], dtype=torch.int32).cuda()
    rows = ((17, cut), (cut, N - 5))
    f32 = dict(out_dtype=torch.float32)
    Y = ssg.grouped_mm(X, W, offs, **f32)
    for e, (lo, hi) in enumerate(rows):
        assert torch.equal(Y[lo:hi], outer(a[lo:hi], W[e].float() @ b, torch.float32))
    assert (Y[:17] == 0).all() and (Y[N - 5:] == 0).all()
    del Y
    dW = ssg.grouped_mm_dw(dY, X, offs, **f32)
    for e, (lo, hi) in enumerate(rows):
        total = (a[lo:hi] * c[lo:hi]).double().sum().float()
        assert total.abs() * 4 < 1 << 24
        assert torch.equal(dW[e], outer(d, b, torch.float32) * total)
    del X
    dX = ssg.grouped_mm_dx(dY, W, offs)
    for e, (lo, hi) in enumerate(rows):
        want = d @ W[e].float()
        assert want.abs().max() <= 256
        for at in (lo, hi - 20_000):
            assert torch.equal(dX[at:at + 20_000].float(), outer(c[at:at + 20_000], want, torch.float32))
    assert (dX[:17] == 0).all() and (dX[N - 5:] == 0).all()


@pytest.mark.parametrize("x", ["bf16", "mx4"])
def test_mx4_weights_and_tokens_past_32_bits(x):
    K, M = 4096, 66
    N = ((1 << 32) // (K // 2 if x == "mx4" else 2 * K)) + 30_000
    a, b = cycle(N, 3, -1), cycle(K, 5, -2)
    X = outer(a, b)
    W = outer(cycle(M, 3, -1), cycle(K, 3, 0))
    we, ws = ssg.mx4_quantize(W)
    offs = torch.tensor([0, 20_000, N], dtype=torch.int32).cuda()
    want = W.float() @ b
    kw = {}
    if x == "mx4":
        X, kw["xscales"] = ssg.mx4_quantize(X)
    for Y in (lambda: ssg.mm_mx4(X, we, ws, **kw),
              lambda: ssg.grouped_mm_mx4(X, we[None].expand(2, *we.shape), ws[None].expand(2, *ws.shape), offs, **kw)):
        assert torch.equal(Y(), outer(a, want, torch.float32))


def test_quantise_past_32_bits():
    # more pieces of 8 elements than one launch counts
    K = 4096
    R = (1 << 30) // (K // 8) + 1000
    X = outer(cycle(R, 7, -3), cycle(K, 5, -2))
    e, s = ssg.mx4_quantize(X)
    for lo in (0, (1 << 30) // (K // 8) - 500, R - 700):
        some = slice(lo, lo + 700)
        e1, s1 = ssg.mx4_quantize(X[some])
        assert torch.equal(e[some], e1) and torch.equal(s[some], s1)
    del X
    back = ssg.mx4_dequantize(e, s, K, dtype=torch.bfloat16)
    for lo in (0, (1 << 30) // (K // 8) - 500, R - 700):
        want = outer(cycle(R, 7, -3)[lo:lo + 700], cycle(K, 5, -2))
        assert torch.equal(back[lo:lo + 700], want)


@pytest.mark.parametrize("E,N", [(65, 300), (300, 2000), (1000, 37), (4097, 9000)])
def test_many_experts(E, N):
    M, K = 24, 40
    g = torch.Generator().manual_seed(E)
    ends, _ = torch.randint(0, N + 1, (E + 1,), generator=g).sort()
    offs = ends.to(torch.int32)
    X, W, dY = D.randn((N, K), "f16", 1), D.randn((E, M, K), "f16", 2, 0.1), D.randn((N, M), "f16", 3)
    x, w, d = X.double().numpy(), W.double().numpy(), dY.double().numpy()
    most = int((offs[1:] - offs[:-1]).max())
    D.check(ssg.grouped_mm(X.cuda(), W.cuda(), offs.cuda()), *D.grouped(x, w, offs), K, "Y")
    D.check(ssg.grouped_mm_dx(dY.cuda(), W.cuda(), offs.cuda()), *D.grouped_dx(d, w, offs), M, "dX")
    D.check(ssg.grouped_mm_dw(dY.cuda(), X.cuda(), offs.cuda()), *D.grouped_dw(d, x, offs), most, "dW")
    e, s = D.random_mx4((E, M, K), 4)
    xe, xs = D.random_mx4((N, K), 5, 120, 130)
    w4, x4 = D.mx4_values(e, s, K), D.mx4_values(xe, xs, K)
    e, s, xe, xs = (torch.from_numpy(t).cuda() for t in (e, s, xe, xs))
    D.check(ssg.grouped_mm_mx4(X.cuda(), e, s, offs.cuda()), *D.grouped(x, w4, offs), K, "mx4 weights")
    D.check(ssg.grouped_mm_mx4(xe, e, s, offs.cuda(), xscales=xs), *D.grouped(x4, w4, offs), K, "mx4 x mx4")
