"""The expert-grouped 16-bit products and their gradients through the public
calls, against 64-bit definitions."""
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


def case(dt, sizes, M, K, seed, first=0, extra=0):
    E, N = len(sizes), first + sum(sizes) + extra
    X, W, dY = D.randn((N, K), dt, seed), D.randn((E, M, K), dt, seed + 1, 0.1), D.randn((N, M), dt, seed + 2)
    return X, W, dY, D.offsets(sizes, first)


# (sizes, M, K): single tokens; empty experts; around the kernels' borders; odd lengths; many experts; one expert
CASES = [([1], 16, 32), ([0, 1, 0], 8, 8), ([2, 0, 1], 100, 72), ([16, 17], 40, 1000), ([33, 0, 64, 31], 264, 136),
         ([65, 63, 128, 129], 136, 264), ([300, 0, 2], 520, 400), ([7] * 40, 33, 35), ([50, 1, 90], 77, 101),
         ([257], 300, 513), ([0, 0], 24, 40), ([40, 60], 1, 1), ([500, 24, 0, 300], 129, 1023),
         ([70, 45], 70, 1002), ([3, 2], 262, 34), ([130, 0, 260], 390, 86), ([1, 0, 3], 20, 5000)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("which", range(len(CASES)))
def test_forward_and_gradients(dt, which):
    sizes, M, K = CASES[which]
    X, W, dY, offs = case(dt, sizes, M, K, which)
    x, w, d = (t.double().numpy() for t in (X, W, dY))
    Xg, Wg, dYg, og = X.cuda(), W.cuda(), dY.cuda(), offs.cuda()
    for out in (dt, "f32"):
        o = D.TORCH[out]
        D.check(ssg.grouped_mm(Xg, Wg, og, out_dtype=o), *D.grouped(x, w, offs), K, "Y %s" % out)
        D.check(ssg.grouped_mm_dx(dYg, Wg, og, out_dtype=o), *D.grouped_dx(d, w, offs), M, "dX %s" % out)
        D.check(ssg.grouped_mm_dw(dYg, Xg, og, out_dtype=o), *D.grouped_dw(d, x, offs), max(sizes), "dW %s" % out)


@pytest.mark.parametrize("rows", [1, 40])
def test_rows_of_no_expert(rows):
    X, W, dY, offs = case("bf16", [rows, 0, 3 * rows], 90, 72, 5, first=30, extra=25)
    Xg, Wg, dYg, og = X.cuda(), W.cuda(), dY.cuda(), offs.cuda()
    Y, dX, dW = ssg.grouped_mm(Xg, Wg, og), ssg.grouped_mm_dx(dYg, Wg, og), ssg.grouped_mm_dw(dYg, Xg, og)
    for t in (Y, dX):
        assert (t[:30] == 0).all() and (t[30 + 4 * rows:] == 0).all() and (t[30:30 + rows] != 0).any()
    D.check(dW, *D.grouped_dw(dY.double().numpy(), X.double().numpy(), offs), 3 * rows, "dW")
    assert (dW[1] == 0).all()


def test_rows_of_no_expert_may_hold_nan():
    # nobody's rows, and another expert's, must not reach an expert's gradient
    X, W, dY, offs = case("f16", [20, 70], 40, 56, 6, first=10, extra=10)
    for t in (X, dY):
        t[:10] = float("nan")
        t[100:] = float("inf")
    X[35], dY[35] = float("nan"), float("nan")            # expert 1
    Xg, Wg, dYg, og = X.cuda(), W.cuda(), dY.cuda(), offs.cuda()
    dW = ssg.grouped_mm_dw(dYg, Xg, og)
    assert torch.isfinite(dW[0]).all() and torch.isnan(dW[1]).all()
    Y = ssg.grouped_mm(Xg, Wg, og)
    assert (Y[:10] == 0).all() and torch.isnan(Y[35]).all()
    assert torch.isfinite(Y[10:35]).all() and torch.isfinite(Y[36:100]).all()


def test_strided_operands():
    sizes, M, K = [10, 70, 0, 30], 120, 136
    X, W, dY, offs = case("bf16", sizes, M, K, 8)
    for pad in (3, 8):                                    # rows off and on 16-byte alignment
        Xb = torch.full((110, K + 2 * pad), float("nan"), dtype=torch.bfloat16).cuda()
        Wb = torch.full((4, M + 5, K + 3 * pad), float("nan"), dtype=torch.bfloat16).cuda()
        Db = torch.full((110, M + pad), float("nan"), dtype=torch.bfloat16).cuda()
        Xv, Wv, Dv = Xb[:, pad:pad + K], Wb[:, 2:2 + M, pad:pad + K], Db[:, :M]
        Xv.copy_(X)
        Wv.copy_(W)
        Dv.copy_(dY)
        x, w, d = (t.double().numpy() for t in (X, W, dY))
        Y = torch.full((110, M + 7), 7.0).cuda()
        ssg.ssg_grouped_mm(Xv, Wv, offs.cuda(), Y[:, 2:2 + M])
        D.check(Y[:, 2:2 + M], *D.grouped(x, w, offs), K, "Y")
        assert (Y[:, :2] == 7).all() and (Y[:, 2 + M:] == 7).all()
        D.check(ssg.grouped_mm_dx(Dv, Wv, offs.cuda()), *D.grouped_dx(d, w, offs), M, "dX")
        dW = torch.full((4, M + 1, K + 6), 7.0).cuda()
        ssg.ssg_grouped_mm_dw(Dv, Xv, offs.cuda(), dW[:, :M, 3:3 + K])
        D.check(dW[:, :M, 3:3 + K], *D.grouped_dw(d, x, offs), 70, "dW")
        assert (dW[:, M:] == 7).all() and (dW[:, :, :3] == 7).all() and (dW[:, :, 3 + K:] == 7).all()


def test_no_experts_and_no_rows():
    og = torch.zeros(1, dtype=torch.int32).cuda()
    X, dY = torch.ones(5, 16, dtype=torch.float16).cuda(), torch.ones(5, 24, dtype=torch.float16).cuda()
    W = torch.empty(0, 24, 16, dtype=torch.float16).cuda()
    assert (ssg.grouped_mm(X, W, og) == 0).all() and (ssg.grouped_mm_dx(dY, W, og) == 0).all()
    assert ssg.grouped_mm_dw(dY, X, og).shape == (0, 24, 16)
    og = torch.zeros(4, dtype=torch.int32).cuda()
    W = torch.ones(3, 24, 16, dtype=torch.float16).cuda()
    assert ssg.grouped_mm(X[:0], W, og).shape == (0, 24)
    assert (ssg.grouped_mm_dw(dY[:0], X[:0], og) == 0).all()
    assert (ssg.grouped_mm(X, W, og) == 0).all()


def test_gradients_against_differences():
    # loss = sum of c * Y: its difference quotients in the direction of every
    # input, by 64-bit forward products of the inputs the kernels saw
    sizes, M, K = [5, 0, 40], 24, 32
    X, W, dY, offs = case("bf16", sizes, M, K, 11)
    x, w, c = (t.double().numpy() for t in (X, W, dY))
    rng = np.random.default_rng(12)
    ux, uw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
    h = 2.0 ** -10

    def loss(a, b):
        return float((c * D.grouped(a, b, offs)[0]).sum())

    dX = ssg.grouped_mm_dx(dY.cuda(), W.cuda(), offs.cuda(), out_dtype=torch.float32).double().cpu().numpy()
    dW = ssg.grouped_mm_dw(dY.cuda(), X.cuda(), offs.cuda(), out_dtype=torch.float32).double().cpu().numpy()
    # the loss is linear in each input: the quotients are exact up to 64-bit
    # cancellation, and the kernels are off by (length + 16) 2^-23 of the magnitudes
    for got, u, quotient, mag, length in [
            (dX, ux, (loss(x + h * ux, w) - loss(x - h * ux, w)) / (2 * h), D.grouped_dx(c, w, offs)[1], M),
            (dW, uw, (loss(x, w + h * uw) - loss(x, w - h * uw)) / (2 * h), D.grouped_dw(c, x, offs)[1], 40)]:
        bound = (length + 16) * 2.0 ** -23 * (np.abs(u) * mag).sum()
        assert abs((got * u).sum() - quotient) <= bound


def test_expert_weights_past_32_bits():
    # the last expert's rows start more than 2^32 bytes into the stack
    E, M, K = 5, 16384, 32768
    W = torch.zeros(E, M, K, dtype=torch.bfloat16, device="cuda")
    W[4, :, :64] = 1.0
    W[4, M - 1, K - 8:] = 2.0
    X = torch.ones(3, K, dtype=torch.bfloat16, device="cuda")
    offs = D.offsets([1, 0, 0, 0, 2]).cuda()
    Y = ssg.grouped_mm(X, W, offs, out_dtype=torch.float32)
    want = torch.full((3, M), 64.0, device="cuda")
    want[0] = 0
    want[1:, M - 1] += 16
    assert torch.equal(Y, want)
    dX = ssg.grouped_mm_dx(torch.ones(3, M, dtype=torch.bfloat16, device="cuda"), W, offs, out_dtype=torch.float32)
    want = torch.zeros(3, K, device="cuda")
    want[1:, :64] = M
    want[1:, K - 8:] = 2
    assert torch.equal(dX, want)


def test_same_bits_each_call_and_on_another_stream():
    X, W, dY, offs = case("f16", [100, 3, 0, 77], 264, 328, 13)
    Xg, Wg, dYg, og = X.cuda(), W.cuda(), dY.cuda(), offs.cuda()
    calls = [lambda s=None: ssg.grouped_mm(Xg, Wg, og, stream=s), lambda s=None: ssg.grouped_mm_dx(dYg, Wg, og, stream=s),
             lambda s=None: ssg.grouped_mm_dw(dYg, Xg, og, stream=s)]
    side = torch.cuda.Stream()
    for f in calls:
        a = f()
        torch.cuda.synchronize()
        for _ in range(3):
            b = f(side)
            side.synchronize()
            assert torch.equal(a, b)


def test_captured_step_replays():
    # forward, both gradients and a quantised product in one graph, replayed
    # with new inputs and offsets between eager runs
    sizes = [[40, 0, 24, 36], [1, 90, 0, 9], [0, 0, 0, 100]]
    K, M, N = 136, 72, 100
    W = D.randn((4, M, K), "bf16", 1, 0.1).cuda()
    We, Ws = ssg.mx4_quantize(W)
    X, dY = torch.zeros(N, K, dtype=torch.bfloat16).cuda(), torch.zeros(N, M, dtype=torch.bfloat16).cuda()
    offs = torch.zeros(5, dtype=torch.int32).cuda()

    def step():
        xe, xs = ssg.mx4_quantize(X)
        return (ssg.grouped_mm(X, W, offs), ssg.grouped_mm_dx(dY, W, offs), ssg.grouped_mm_dw(dY, X, offs),
                ssg.grouped_mm_mx4(X, We, Ws, offs), ssg.grouped_mm_mx4(xe, We, Ws, offs, xscales=xs))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i, sz in enumerate(sizes + sizes):
        X.copy_(D.randn((N, K), "bf16", 20 + i))
        dY.copy_(D.randn((N, M), "bf16", 40 + i))
        offs.copy_(D.offsets(sz))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_compiled_and_python_marshalling_agree():
    # the compiled path takes the call without a stream, the Python one the call
    # with the current stream named: the same bits, also where a workspace is needed
    cur = torch.cuda.current_stream()
    for dt, sizes, M, K in [("bf16", [3, 0, 5], 72, 64), ("f16", [90, 40], 264, 1001), ("bf16", [30], 512, 2048)]:
        X, W, dY, offs = case(dt, sizes, M, K, 3)
        Xg, Wg, dYg, og = X.cuda(), W.cuda(), dY.cuda(), offs.cuda()
        for f, a in [(ssg.grouped_mm, (Xg, Wg, og)), (ssg.grouped_mm_dx, (dYg, Wg, og)), (ssg.grouped_mm_dw, (dYg, Xg, og))]:
            for out in (None, torch.float32):
                assert torch.equal(f(*a, out_dtype=out), f(*a, out_dtype=out, stream=cur))
        e, s = ssg.mx4_quantize(Wg)
        e1, s1 = ssg.mx4_quantize(Xg)
        e2, s2 = ssg.mx4_quantize(Xg, stream=cur)
        assert torch.equal(e1, e2) and torch.equal(s1, s2)
        assert torch.equal(ssg.mx4_dequantize(e1, s1, K), ssg.mx4_dequantize(e1, s1, K, stream=cur))
        assert torch.equal(ssg.grouped_mm_mx4(Xg, e, s, og), ssg.grouped_mm_mx4(Xg, e, s, og, stream=cur))
        assert torch.equal(ssg.mm_mx4(Xg, e[0], s[0]), ssg.mm_mx4(Xg, e[0], s[0], stream=cur))
        if K % 32 == 0:
            assert torch.equal(ssg.mm_mx4(e1, e[0], s[0], xscales=s1), ssg.mm_mx4(e1, e[0], s[0], xscales=s1, stream=cur))


def test_refusals_on_the_device():
    X, W, dY, offs = (t.cuda() for t in case("f16", [4, 4], 24, 32, 1))
    e, s = ssg.mx4_quantize(W)

    def status(f, *a, **k):
        with pytest.raises(ssg.SsgError) as err:
            f(*a, **k)
        return err.value.status

    assert status(ssg.grouped_mm, X, W, offs.long()) == 4
    assert status(ssg.grouped_mm, X, W, offs[:2]) == 2
    assert status(ssg.grouped_mm, X, W, offs, out_dtype=torch.bfloat16) == 4
    assert status(ssg.grouped_mm, X, W.transpose(1, 2), offs) in (2, 3)
    assert status(ssg.grouped_mm, X.t().contiguous().t(), W, offs) == 3
    assert status(ssg.grouped_mm_dx, X, W, offs) == 2
    assert status(ssg.grouped_mm_dw, dY, X[:4], offs) == 2
    assert status(ssg.grouped_mm_mx4, X, e, s[:, :, :0], offs) == 2
    assert status(ssg.mm_mx4, X, e[0], s[0], out_dtype=torch.bfloat16) == 4
    assert status(ssg.mx4_quantize, X.double()) == 4


@pytest.mark.parametrize("M,K", [(70, 70), (72, 1002), (300, 262), (66, 65)])
@pytest.mark.parametrize("rows", [3, 60, 300])
def test_a_row_of_nan_stays_in_its_row(M, K, rows):
    # lengths that end inside a 16-byte piece of a row: what the piece brings of
    # the next row must not reach this one's sums
    sizes = [rows, rows + 7]
    X, W, dY, offs = case("bf16", sizes, M, K, 9)
    N = 2 * rows + 7
    X[1] = float("nan")
    W[0, 5] = float("nan")
    dY[2] = float("nan")
    W2 = W.clone()
    W2[0, 5] = 1.0
    og = offs.cuda()
    Y = ssg.grouped_mm(X.cuda(), W.cuda(), og).float().cpu()
    want = torch.zeros(N, M, dtype=torch.bool)
    want[1] = True
    want[:rows, 5] = True
    assert torch.equal(torch.isnan(Y), want)
    dX = ssg.grouped_mm_dx(dY.cuda(), W2.cuda(), og).float().cpu()
    want = torch.zeros(N, K, dtype=torch.bool)
    want[2] = True
    assert torch.equal(torch.isnan(dX), want)
    X[1] = 0
    X[rows:, K - 1] = float("inf")
    dY[2] = 0
    dY[rows:] = dY[rows:].abs() + 1
    dW = ssg.grouped_mm_dw(dY.cuda(), X.cuda(), og).float().cpu()
    assert torch.isfinite(dW[0]).all() and torch.isfinite(dW[1, :, :K - 1]).all()
    assert (dW[1, :, K - 1] == float("inf")).all()


# tiles of the largest size, its halves and quarters, in whole and partly filled rounds
@pytest.mark.parametrize("sizes,M,K", [([900, 0, 1500, 333], 2304, 1058), ([2100], 4096, 512), ([257, 255, 256], 1024, 520),
                                       ([3000, 100, 700], 2560, 264)])
def test_large_products(sizes, M, K):
    X, W, dY, offs = case("bf16", sizes, M, K, 17)
    Xg, Wg, dYg, og = X.cuda(), W.cuda(), dY.cuda(), offs.cuda()
    x, w, d = Xg.double(), Wg.double(), dYg.double()
    e, s = ssg.mx4_quantize(Wg)
    xe, xs = ssg.mx4_quantize(Xg)
    wq, xq = ssg.mx4_dequantize(e, s, K).double(), ssg.mx4_dequantize(xe, xs, K).double()
    got = {"Y": ssg.grouped_mm(Xg, Wg, og), "dX": ssg.grouped_mm_dx(dYg, Wg, og, out_dtype=torch.float32),
           "dW": ssg.grouped_mm_dw(dYg, Xg, og), "w4": ssg.grouped_mm_mx4(Xg, e, s, og),
           "mx": ssg.grouped_mm_mx4(xe, e, s, og, xscales=xs, out_dtype=torch.bfloat16)}
    for i, a, b in D.segments(offs, X.shape[0]):
        parts = {"Y": (x[a:b], w[i].t(), K), "dX": (d[a:b], w[i], M), "dW": (d[a:b].t(), x[a:b], b - a),
                 "w4": (x[a:b], wq[i].t(), K), "mx": (xq[a:b], wq[i].t(), K)}
        for name, (l, r, n) in parts.items():
            l, r = l.contiguous(), r.contiguous()
            out = got[name][i] if name == "dW" else got[name][a:b]
            D.check(out, (l @ r).cpu().numpy(), (l.abs() @ r.abs()).cpu().numpy(), n, "%s of expert %d" % (name, i))
