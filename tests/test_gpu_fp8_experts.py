"""The operators around experts and of 8-bit floats together: the example's
gradients against the formulas, an 8-bit layer against its definition, served
from a captured graph, and operands of more than 2^32 bytes."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from examples import fp8_experts as ex
from tests import _experts as D
from tests import _fp8 as F

pytestmark = pytest.mark.gpu


def np64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------- gradients

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k,C", [(1, 4, 2, 8), (60, 12, 3, 130), (33, 64, 6, 64)])
def test_gradients_through_route_gather_and_combine(score, N, E, k, C):
    """out[n] = sum_j w[n, j] r[pos[n, j]] x[n] with numbers r for the rows, in fp32: a
    weight is off by (E + 16 + 2 range) steps of 2^-23 (as the routing's tests derive),
    a sum of n products by n, each product by one more."""
    l, x = D.randn((N, E), "f32", 1), D.randn((N, C), "f32", 2)
    if N > 2:
        l[-1] = -float("inf")                                   # a padded token
        l[0, 1:] = -float("inf")                                # one with a single expert
    bias, g = D.randn((E,), "f32", 3), D.randn((N, C), "f32", 4)
    lg, xg = l.cuda().requires_grad_(), x.cuda().requires_grad_()
    w, e = ex.Route.apply(lg, k, score, bias.cuda(), 1, 1)
    offs, rows, pos = ssg.expert_order(e, E)
    r = D.randn((N * k, 1), "f32", 5)
    out = ex.Combine.apply(ex.Gather.apply(xg, pos, rows) * r.cuda(), pos, rows, w)
    out.backward(g.cuda())

    l64, x64, g64, r64 = np64(l), np64(x), np64(g), np64(r)[:, 0]
    w64, e64 = D.route(l64, k, score=score, bias=np64(bias))
    assert np.array_equal(e.cpu().numpy(), e64)
    _, _, p64 = D.order(e64, E)
    s = np.where(p64 >= 0, r64[p64], 0.0)                       # number of a pair's row
    fin = l64[np.isfinite(l64)]
    bound = (E + 16 + 2 * np.ptp(fin)) * 2.0 ** -23 if fin.size else 0.0
    f = (w64 * s).sum(1, keepdims=True)
    fm = (w64 * np.abs(s)).sum(1, keepdims=True)
    off = bound + (k + 3) * 2.0 ** -23
    D.close(out.detach(), f * x64, off * fm * np.abs(x64), "out")
    D.close(xg.grad, f * g64, off * fm * np.abs(g64), "dx")
    # dw[n, j] = s <g, x>
    dw = s * (g64 * x64).sum(1, keepdims=True)
    dwm = np.abs(s) * (np.abs(g64) * np.abs(x64)).sum(1, keepdims=True)
    ref, mag = D.route_grad(dw, l64, e64, score=score)
    _, whole = D.route_grad(dwm, l64, e64, score=score)
    D.close(lg.grad, ref, 4 * bound * mag + (C + 3) * 2.0 ** -23 * whole + 2.0 ** -120, "dlogits")
    if N > 2:
        assert (lg.grad[-1] == 0).all() and (xg.grad[-1] == 0).all() and (out[-1] == 0).all()


@pytest.mark.parametrize("N,M,K", [(1, 24, 40), (70, 130, 300), (300, 256, 128)])
def test_gradients_of_the_8_bit_linear(N, M, K):
    x, w, g = (D.randn(n, "f32", i) for i, n in enumerate(((N, K), (M, K), (N, M))))
    xg, wg = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = ex.Fp8Linear.apply(xg, wg)
    y.backward(g.cuda())
    v = lambda a, block=1: F.values(*F.quantize(a, block))
    x64, w64, g64 = np64(x), np64(w), np64(g)
    for got, a, b in ((y.detach(), v(x64), v(w64, 128).T), (xg.grad, v(g64), v(w64.T, 128).T), (wg.grad, v(g64.T), v(x64.T).T)):
        F.check(got, a @ b, np.abs(a) @ np.abs(b), a.shape[1], "linear")
    # only what is asked for
    frozen = w.cuda()
    assert torch.equal(torch.autograd.grad(ex.Fp8Linear.apply(xg, frozen), xg, g.cuda())[0], xg.grad)


def test_second_gradients_are_an_error():
    x = D.randn((4, 8), "f32", 1).cuda().requires_grad_()
    w = D.randn((4, 8), "f32", 2).cuda().requires_grad_()
    for f in (lambda: ex.Fp8Linear.apply(x, w), lambda: ex.Route.apply(x, 2, "softmax", None, 1, 1)[0]):
        d, = torch.autograd.grad(f().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            d.sum().backward()


# ---------------------------------------------------------------- an 8-bit layer

@pytest.mark.parametrize("N", [1, 16, 300])
def test_8_bit_experts_against_the_formula(N):
    """One grouped product by 8-bit weights between the gather and the sums: the
    product's bound (of its fp32 sums, the 8-bit instruction and the output), half a
    step of bf16 for its output, and the weights' and sums' steps."""
    E, k, K, M = 16, 4, 200, 96
    l, X, W = D.randn((N, E), "bf16", 1), D.randn((N, K), "bf16", 2), D.randn((E, M, K), "bf16", 3)
    if N > 4:
        l[N - 3:] = -float("inf")
    weights, e = ssg.route(l.cuda(), k)
    offs, rows, pos = ssg.expert_order(e, E)
    w8, s8 = ssg.fp8_quantize(W.cuda(), block=128)
    Y = ssg.grouped_mm_fp8(ssg.expert_gather(X.cuda(), pos, rows), w8, s8, offs, out_dtype=torch.bfloat16)
    O = ssg.expert_combine(Y, pos, weights, out_dtype=torch.float32)
    w64, e64 = D.route(np64(l), k)
    assert np.array_equal(e.cpu().numpy(), e64)
    cx, sx = F.quantize(np64(X))
    xv = F.values(cx, sx)
    ref, tol = np.zeros((N, M)), np.zeros((N, M))
    for i in range(E):
        n, j = np.nonzero(e64 == i)
        if not n.size:
            continue
        cw, sw = F.quantize(np64(W)[i], 128)
        wv = F.values(cw, sw)
        y, m = xv[n] @ wv.T, np.abs(xv[n]) @ np.abs(wv).T
        t = (K + F.blocks(K) + 16) * 2.0 ** -23 * m + F.coarse(xv[n], wv, sx[n], sw)
        t = t + (np.abs(y) + t) * 2.0 ** -8
        share = w64[n, j][:, None]
        np.add.at(ref, n, share * y)
        np.add.at(tol, n, share * (t + (E + 16 + 2 * 16 + k) * 2.0 ** -23 * (np.abs(y) + t)))
    D.close(O, ref, tol, "layer")
    if N > 4:
        assert (O[N - 3:] == 0).all()


def test_serving_replayed_from_graphs():
    # two graphs of one layer, replayed in turn with eager work between
    layer = ex.Layer(8, 256, 384, top=2, score="sigmoid", groups=4, top_groups=2)
    layer.quantise()
    tokens = (1, 48)
    x = [torch.empty(n, 256, dtype=torch.bfloat16).cuda() for n in tokens]

    def fill(seed):
        for i, t in enumerate(x):
            t.copy_(D.randn(tuple(t.shape), "bf16", seed + i))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in x:
            layer.serve(t)
    torch.cuda.current_stream().wait_stream(side)
    graphs, out = [torch.cuda.CUDAGraph() for _ in x], []
    for graph, t in zip(graphs, x):
        with torch.cuda.graph(graph):
            out.append(layer.serve(t))
    for seed in (10, 20, 30):
        fill(seed)
        want = [layer.serve(t).clone() for t in x]
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_example_runs():
    loss = ex.main(["--experts", "8", "--width", "256", "--hidden", "384", "--tokens", "200", "--steps", "3"])
    assert np.isfinite(loss)


# ---------------------------------------------------------------- more than 2^32 bytes

def test_rows_past_32_bits():
    N, k, C, E = 70000, 8, 4096, 8                              # 4.6 GB of rows
    assert N * k * C * 2 > 1 << 32
    X = torch.randn(N, C, device="cuda", dtype=torch.bfloat16)
    e = torch.stack([torch.randperm(E, device="cuda") for _ in range(64)]).int()[torch.arange(N, device="cuda") % 64]
    offs, rows, pos = ssg.expert_order(e.contiguous(), E)
    assert (offs.cpu() == torch.arange(E + 1) * N).all()
    Y = ssg.expert_gather(X, pos, rows)
    some = torch.tensor([0, 1, N * k // 2, N * k - 70001, N * k - 2, N * k - 1], device="cuda")
    assert torch.equal(Y[some], X[(rows[some] // k).long()])
    w = torch.full((N, k), 0.125, device="cuda")                # powers of two: sums are exact
    assert torch.equal(ssg.expert_combine(Y, pos, w), X)
    dY, dw = ssg.expert_combine_backward(X, Y, pos, rows, w)
    assert torch.equal(dY[some], X[(rows[some] // k).long()] * 0.125)
    last = X[-1].double()
    assert ((dw[-1].double() - (last * last).sum()).abs() <= (C + 1) * 2.0 ** -23 * (last * last).sum()).all()


def test_quantising_past_32_bits():
    R, K = 600000, 4096                                         # 4.9 GB
    A = torch.empty(R, K, device="cuda", dtype=torch.bfloat16)
    A.view(-1, 128).copy_(torch.randn(1, 128, device="cuda").bfloat16() + torch.arange(R * K // 128, device="cuda")[:, None] % 97)
    end = 256
    for block in (1, 128):
        e, s = ssg.fp8_quantize(A, block=block)
        tail = A[R // 128 * 128 - end:]
        te, ts = ssg.fp8_quantize(tail, block=block)
        assert torch.equal(e[-tail.shape[0]:].view(torch.uint8), te.view(torch.uint8))
        assert torch.equal(s[-ts.shape[0]:], ts)
        back = ssg.fp8_dequantize(e, s, dtype=torch.bfloat16)
        assert torch.equal(back[-tail.shape[0]:], ssg.fp8_dequantize(te, ts, dtype=torch.bfloat16))
        del back
        t, ts2 = ssg.fp8_quantize(A, block=block, transpose=True)
        tt, _ = ssg.fp8_quantize(tail, block=block, transpose=True)
        assert torch.equal(t[:, -tail.shape[0]:].contiguous().view(torch.uint8), tt.contiguous().view(torch.uint8))
        del t, e


def test_products_past_32_bits():
    # an output of 4.9 GB, and the last of 170 experts' weights, 5.7 GB
    N, M, K = 300000, 8192, 128
    X = torch.randn(N, K, device="cuda", dtype=torch.bfloat16)
    w, s = ssg.fp8_quantize(torch.randn(M, K, device="cuda", dtype=torch.bfloat16), block=128)
    Y = ssg.mm_fp8(X, w, s, out_dtype=torch.bfloat16)
    assert torch.equal(Y[-4096:], ssg.mm_fp8(X[-4096:], w, s, out_dtype=torch.bfloat16))
    del Y
    E, M, K = 170, 4096, 8192
    W = torch.zeros(E, M, K, device="cuda", dtype=torch.uint8)
    W[-1] = torch.randint(0, 0x70, (M, K), device="cuda", dtype=torch.uint8)
    W = W.view(torch.float8_e4m3fn)
    S = torch.rand(E, M // 128, K // 128, device="cuda") + 0.5
    for rows in (3, 700):
        X = torch.randn(rows, K, device="cuda", dtype=torch.bfloat16)
        offs = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
        offs[-1] = rows
        got = ssg.grouped_mm_fp8(X, W, S, offs)
        x, xs = ssg.fp8_quantize(X)
        v = ssg.fp8_dequantize(x, xs).double()
        wv = ssg.fp8_dequantize(W[-1], S[-1]).double()
        assert ((got.double() - v @ wv.t()).abs() <= (K + 64 + 16) * 2.0 ** -23 * (v.abs() @ wv.abs().t()) + 2.0 ** -149).all()
