"""8-bit floats with a scale for each block of 128, and their products, through the
public calls, against 64-bit definitions."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _fp8 as D
from tests import _mm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    torch.cuda.init()
    return torch.device("cuda:0")


def np64(t):
    return t.detach().cpu().double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- the format

def same_form(e, s, a64, block):
    codes, scales = D.quantize(a64, block)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scales, equal_nan=True)
    assert np.array_equal(D.codes_of(e) & 0x7F, codes & 0x7F)
    nan = (codes & 0x7F) == 0x7F                         # (a NaN's sign is free)
    assert np.array_equal(D.codes_of(e)[~nan], codes[~nan])
    return codes, scales


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 1), (3, 127), (17, 128), (128, 130), (130, 300), (2, 4100), (257, 16), (300, 513)])
def test_quantize_and_back(dt, block, R, K):
    a = D.randn((R, K), dt, R + K) * torch.exp2(torch.randint(-9, 9, (R, 1))).to(D.TORCH[dt])
    for tr in (False, True):
        e, s = ssg.fp8_quantize(a.cuda(), block=block, transpose=tr)
        a64 = np64(a).T if tr else np64(a)
        assert e.shape == a64.shape and e.dtype == torch.float8_e4m3fn
        codes, scales = same_form(e, s, a64, block)
        v = torch.from_numpy(D.values(codes, scales).astype(np.float32))   # one rounding, of the product
        for out in ("f32", "f16", "bf16"):
            back = ssg.fp8_dequantize(e, s, dtype=D.TORCH[out])
            assert torch.equal(back.cpu(), v.to(D.TORCH[out])), out


def test_quantize_ties_and_neighbours():
    # quotients on the borders of two codes, and the numbers next to them: the scale
    # is a power of two, then any number (where x / scale is on a border only by rounding)
    mids = (D.CODES[:-1] + D.CODES[1:]) / 2
    for top in (448.0, 448.0 * 0.7712345, 3.0e-5, 1.7e30):
        top = np.float32(top)
        s = np.float32(top / np.float32(448))
        x = (mids * np.float64(s)).astype(np.float32)
        near = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf)),
                               D.CODES.astype(np.float32) * s])
        near = np.concatenate([near, -near])
        near = near[np.abs(near) <= top]
        rows = np.zeros((-(-near.size // 127), 128), dtype=np.float32)
        rows[:, 0] = top
        flat = np.zeros(rows.shape[0] * 127, dtype=np.float32)
        flat[:near.size] = near
        rows[:, 1:] = flat.reshape(-1, 127)
        a = torch.from_numpy(rows)
        for block, tr in ((1, False), (1, True), (128, False), (128, True)):
            e, sc = ssg.fp8_quantize((a.t().contiguous() if tr else a).cuda(), block=block, transpose=tr)
            same_form(e, sc, rows.astype(np.float64), block)


def test_quantize_extremes():
    t = torch.finfo(torch.float32)
    inf, nan = float("inf"), float("nan")
    a = torch.zeros(11, 256)
    a[1, 3], a[1, 140] = t.max, -t.max
    a[2, 0], a[2, 133] = t.smallest_normal, t.smallest_normal * 5
    a[3, 1], a[3, 132] = 1e-45, 3e-45
    a[4, 2], a[4, 3] = inf, 1.0
    a[5, 5], a[5, 6] = nan, 2.0
    a[6, 130], a[6, 131] = nan, -inf
    a[7] = -0.0
    a[8, :128] = nan
    a[9] = torch.linspace(-1, 1, 256)
    a[10, 7] = 447.0 * 2.0 ** -126
    for block, tr in ((1, False), (1, True)):
        e, s = ssg.fp8_quantize((a.t().contiguous() if tr else a).cuda(), block=block, transpose=tr)
        same_form(e, s, np64(a), block)
    b = a.clone()
    b[4], b[6] = 0, 0
    for tr in (False, True):
        e, s = ssg.fp8_quantize((b.t().contiguous() if tr else b).cuda(), block=128, transpose=tr)
        same_form(e, s, np64(b), 128)


def test_quantize_strided_stacked_and_guarded():
    wide = D.randn((3, 140, 400), "bf16", 5).cuda()
    a = wide[:, 2:136, 7:7 + 250]
    for block in (1, 128):
        for tr in (False, True):
            e, s = ssg.fp8_quantize(a, block=block, transpose=tr)
            for i in range(3):
                ei, si = ssg.fp8_quantize(a[i].contiguous(), block=block, transpose=tr)
                assert torch.equal(e[i].contiguous().view(torch.uint8), ei.contiguous().view(torch.uint8))
                assert torch.equal(s[i], si)
            R, K = (250, 134) if tr else (134, 250)
            eb = torch.full((3, R, K + 21), 7, dtype=torch.uint8).cuda()
            n = R if block == 1 else D.blocks(R)
            sb = torch.full((3, n, D.blocks(K) + 3), 7.0).cuda()
            ssg.ssg_fp8_quantize(a, eb[:, :, 5:5 + K].view(torch.float8_e4m3fn), sb[:, :, 1:1 + D.blocks(K)], transpose=tr)
            assert torch.equal(eb[:, :, 5:5 + K], e.contiguous().view(torch.uint8)) and torch.equal(sb[:, :, 1:-2], s)
            assert (eb[:, :, :5] == 7).all() and (eb[:, :, 5 + K:] == 7).all()
            assert (sb[:, :, :1] == 7).all() and (sb[:, :, -2:] == 7).all()
            d = torch.full((3, R, K + 9), 7.0).cuda()
            ssg.ssg_fp8_dequantize(eb[:, :, 5:5 + K].view(torch.float8_e4m3fn), sb[:, :, 1:-2], d[:, :, 4:4 + K])
            assert torch.equal(d[:, :, 4:4 + K], ssg.fp8_dequantize(e, s))
            assert (d[:, :, :4] == 7).all() and (d[:, :, 4 + K:] == 7).all()


def test_quantize_refuses_stacks_that_share_places():
    A = D.randn((3, 130, 200), "bf16", 1).cuda()
    e, s = ssg.fp8_quantize(A, block=128)
    one = torch.empty(130, 200, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn)
    for elems, scales in ((one.expand(3, 130, 200), s), (e, s[:1].expand(3, 2, 2))):
        with pytest.raises(ssg.SsgError):
            ssg.ssg_fp8_quantize(A, elems, scales)
    with pytest.raises(ssg.SsgError):
        ssg.ssg_fp8_dequantize(e, s, torch.empty(130, 200).cuda().expand(3, 130, 200))
    # matrices between each other's rows share none
    mixed = torch.zeros(130, 3, 208, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn).transpose(0, 1)[..., :200]
    ssg.ssg_fp8_quantize(A, mixed, s)
    assert torch.equal(mixed.contiguous().view(torch.uint8), e.contiguous().view(torch.uint8))


def test_quantize_empty():
    for shape in ((0, 64), (5, 0), (0, 0), (2, 0, 7), (0, 4, 4)):
        for block in (1, 128):
            e, s = ssg.fp8_quantize(torch.empty(shape).cuda(), block=block)
            assert e.shape == shape and ssg.fp8_dequantize(e, s).shape == shape


# ---------------------------------------------------------------- products

# (M, K, N): one of everything, single tokens, around 16, 32, 64, 128 and 256 rows, lengths
# that end inside a dword, 16 bytes and a block
SHAPES = [(1, 1, 1), (16, 128, 1), (33, 100, 3), (130, 4096, 1), (300, 1000, 16), (64, 512, 17), (96, 516, 32),
          (257, 160, 33), (260, 333, 65), (500, 1024, 100), (513, 264, 257), (40, 2112, 300), (129, 31, 600),
          (256, 384, 256), (1000, 131, 130)]


def activations(x, N, K, seed, **span):
    """(arguments, float64 values, scales) of activations of type x."""
    if x == "e4m3":
        c, s = D.random_fp8(N, K, seed, **span)
        return dict(X=D.elements(c), xscales=dev(s)), D.values(c, s.astype(np.float64)), s
    a = D.randn((N, K), x, seed)
    c, s = D.quantize(np64(a))
    return dict(X=a.cuda()), D.values(c, s), s


@pytest.mark.parametrize("x", ["e4m3", "bf16", "f16", "f32"])
@pytest.mark.parametrize("wblock", [1, 128])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_mm_fp8(x, wblock, M, K, N):
    ax, xv, xs = activations(x, N, K, M + K)
    c, s = D.random_fp8(M, K, N + K, wblock)
    wv = D.values(c, s.astype(np.float64))
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    loss = D.coarse(xv, wv, xs, s)
    for out in ("f32", "bf16", "f16"):
        Y = ssg.mm_fp8(ax["X"], D.elements(c), dev(s), xscales=ax.get("xscales"), out_dtype=D.TORCH[out])
        assert Y.dtype == D.TORCH[out]
        if out != "f16" or np.abs(ref).max() < 6e4:
            D.check(Y, ref, mag, K, "mm_fp8 %s -> %s" % (x, out), loss)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_mm_fp8_of_near_magnitudes(M, K, N):
    """Elements of magnitudes 2^-1 to 2^2 less a step: products of 7 fraction bits and
    exponents -2 to 3 are whole multiples of 2^-8, above the cut at 2^(3 - 13), so
    no instruction loses any of them, and 16-bit outputs are held to fp32's bound."""
    lo, hi = (6 << 3), (9 << 3)
    ax, xv, _ = activations("e4m3", N, K, M + K, lo=lo, hi=hi)
    for wblock in (1, 128):
        c, s = D.random_fp8(M, K, N + K, wblock, lo, hi)
        wv = D.values(c, s.astype(np.float64))
        for out in ("f32", "bf16", "f16"):
            Y = ssg.mm_fp8(ax["X"], D.elements(c), dev(s), xscales=ax["xscales"], out_dtype=D.TORCH[out])
            ref = xv @ wv.T
            if out != "f16" or np.abs(ref).max() < 6e4:
                D.check(Y, ref, np.abs(xv) @ np.abs(wv).T, K, "mm_fp8 -> %s" % out)


@pytest.mark.parametrize("sizes,M,K", [([0, 1, 0, 3], 40, 200), ([17, 0, 64, 5, 33], 130, 128), ([300, 1, 257], 257, 333),
                                       ([0, 0], 8, 8), ([90] * 9, 200, 640), ([1] * 20, 33, 100), ([600, 0, 2], 128, 96)])
@pytest.mark.parametrize("x", ["e4m3", "bf16"])
def test_grouped_mm_fp8(x, sizes, M, K):
    # rows before the first and behind the last expert are nobody's
    for first, rest in ((0, 0), (3, 5)):
        N, E = first + sum(sizes) + rest, len(sizes)
        ax, xv, xs = activations(x, N, K, M + K)
        for wblock in (1, 128):
            parts = [D.random_fp8(M, K, N + K + e, wblock) for e in range(E)]
            wv = np.stack([D.values(c, s.astype(np.float64)) for c, s in parts])
            offs = _mm.offsets(sizes, first)
            ref, mag = _mm.grouped(xv, wv, offs.tolist())
            loss = np.zeros_like(ref)
            for e, a, b in _mm.segments(offs.tolist(), N):
                loss[a:b] = D.coarse(xv[a:b], wv[e], xs[a:b], parts[e][1])
            W, S = D.elements(np.stack([c for c, _ in parts])), dev(np.stack([s for _, s in parts]))
            for out in ("f32", "bf16"):
                Y = ssg.grouped_mm_fp8(ax["X"], W, S, offs.cuda(), xscales=ax.get("xscales"), out_dtype=D.TORCH[out])
                D.check(Y, ref, mag, K, "grouped_mm_fp8 %s -> %s" % (x, out), loss)
                assert (Y[:first] == 0).all() and (Y[N - rest:] == 0).all()


@pytest.mark.parametrize("N", [1, 20, 300])
def test_mm_of_quantised_operands_is_the_same_call_by_call(N):
    # rounded in the call or before it, scales by rows or by blocks: the same result
    X, W = D.randn((N, 700), "bf16", 1).cuda(), D.randn((260, 700), "bf16", 2).cuda()
    w, ws = ssg.fp8_quantize(W, block=128)
    x, xs = ssg.fp8_quantize(X)
    want = ssg.mm_fp8(X, w, ws)
    assert torch.equal(ssg.mm_fp8(x, w, ws, xscales=xs), want)
    assert torch.equal(ssg.mm_fp8(x, w, ws, xscales=xs.contiguous()), want)
    assert torch.equal(ssg.mm_fp8(x.contiguous(), w.contiguous(), ws.t().contiguous().t(), xscales=xs), want)
    w1, w1s = ssg.fp8_quantize(W)
    a = ssg.mm_fp8(x, w1, w1s, xscales=xs)
    assert torch.equal(ssg.mm_fp8(x, w1.contiguous(), w1s.contiguous(), xscales=xs), a)
    ones = torch.ones(1, 1).cuda()
    assert torch.equal(ssg.mm_fp8(x, w, ones.expand(3, 6), xscales=ones.expand(N, 6)),
                       ssg.mm_fp8(x, w, torch.ones(3, 6).cuda(), xscales=torch.ones(N, 6).cuda()))


@pytest.mark.parametrize("N", [5, 40, 300])
def test_mm_strided_unaligned_and_guarded(N):
    M, K = 150, 384
    cx, sx = D.random_fp8(N, K, 1)
    cw, sw = D.random_fp8(M, K, 2, 128)
    xv, wv = D.values(cx, sx.astype(np.float64)), D.values(cw, sw.astype(np.float64))
    ref, mag, loss = xv @ wv.T, np.abs(xv) @ np.abs(wv).T, D.coarse(xv, wv, sx, sw)
    for pad in (1, 2, 4, 16):                            # NaN around every operand
        xb = torch.full((N, K + 2 * pad), 0x7F, dtype=torch.uint8).cuda()
        wb = torch.full((M, K + 2 * pad), 0x7F, dtype=torch.uint8).cuda()
        xb[:, pad:pad + K], wb[:, pad:pad + K] = dev(cx), dev(cw)
        sb = torch.full((N, 9), float("nan")).cuda()
        sb[:, 2:5] = dev(sx)
        f = torch.float8_e4m3fn
        Yb = torch.full((N, M + 6), 7.0, dtype=torch.bfloat16).cuda()
        ssg.ssg_mm_fp8(xb.view(f)[:, pad:pad + K], wb.view(f)[:, pad:pad + K], dev(sw), Yb[:, 3:3 + M], xscales=sb[:, 2:5])
        D.check(Yb[:, 3:3 + M], ref, mag, K, "mm_fp8", loss)
        assert (Yb[:, :3] == 7).all() and (Yb[:, 3 + M:] == 7).all()
    for K2 in (383, 381, 260, 129):                      # the rest of a row is not read into the sums
        xb, wb = dev(cx), dev(cw)
        xb[:, K2:], wb[:, K2:] = 0x7F, 0x7F
        nb = D.blocks(K2)
        x2, w2 = D.values(cx[:, :K2], sx[:, :nb].astype(np.float64)), D.values(cw[:, :K2], sw[:, :nb].astype(np.float64))
        Y = ssg.mm_fp8(xb.view(f)[:, :K2], wb.view(f)[:, :K2], dev(sw)[:, :nb], xscales=dev(sx)[:, :nb])
        D.check(Y, x2 @ w2.T, np.abs(x2) @ np.abs(w2).T, K2, "mm_fp8")


def test_mm_nan_and_infinity_stay_in_their_rows():
    for N in (4, 200):
        X, W = D.randn((N, 256), "bf16", 1), D.randn((140, 256), "bf16", 2)
        w, ws = ssg.fp8_quantize(W.cuda(), block=128)
        want = ssg.mm_fp8(X.cuda(), w, ws)
        X[1, 7], X[3, 200] = float("nan"), float("inf")
        Y = ssg.mm_fp8(X.cuda(), w, ws)
        assert torch.isnan(Y[1]).all() and torch.isnan(Y[3]).all()
        keep = [n for n in range(N) if n not in (1, 3)]
        assert torch.equal(Y[keep], want[keep])


def test_products_of_nothing():
    f = torch.float8_e4m3fn
    for N, M, K in ((0, 8, 64), (4, 0, 64), (4, 8, 0), (300, 8, 0)):
        Y = ssg.mm_fp8(torch.empty(N, K).half().cuda(), torch.empty(M, K).cuda().to(f),
                       torch.empty(D.blocks(M), D.blocks(K)).cuda())
        assert Y.shape == (N, M) and (Y == 0).all()
    offs = torch.zeros(1, dtype=torch.int32).cuda()      # no experts: nobody's rows
    Y = ssg.grouped_mm_fp8(torch.ones(5, 16).half().cuda(), torch.empty(0, 8, 16).cuda().to(f), torch.empty(0, 1, 1).cuda(), offs)
    assert Y.shape == (5, 8) and (Y == 0).all()


def test_offsets_out_of_range():
    f = torch.float8_e4m3fn
    w, ws = ssg.fp8_quantize(D.randn((3, 40, 130), "bf16", 1).cuda(), block=128)
    for N in (7, 200):
        X = D.randn((N, 130), "bf16", 2).cuda()
        for offs in ([-5, 3, 2 ** 31 - 1, 4], [5, 2, 9, 1], [-3, -2, -1, -2 ** 31]):
            Yb = torch.full((N + 2, 40), 7.0).cuda()
            ssg.ssg_grouped_mm_fp8(X, w, ws, torch.tensor(offs, dtype=torch.int32).cuda(), Yb[1:-1])
            assert (Yb[0] == 7).all() and (Yb[-1] == 7).all()


# ---------------------------------------------------------------- a training step, streams, graphs

@pytest.mark.parametrize("N,M,K", [(1, 8, 16), (37, 130, 257), (300, 260, 384), (513, 96, 1000)])
def test_gradients_of_a_linear(N, M, K):
    """Y = X W^T, dX and dW from operands quantised along the contraction of each,
    against the products of the definition's values."""
    X, W, dY = D.randn((N, K), "bf16", 1), D.randn((M, K), "bf16", 2, 0.02), D.randn((N, M), "bf16", 3)
    w, ws = ssg.fp8_quantize(W.cuda(), block=128)
    wt, wts = ssg.fp8_quantize(W.cuda(), block=128, transpose=True)
    xt, xts = ssg.fp8_quantize(X.cuda(), transpose=True)
    dyt, dyts = ssg.fp8_quantize(dY.cuda(), transpose=True)
    w64 = D.values(*D.quantize(np64(W), 128))
    x64, dy64 = D.values(*D.quantize(np64(X))), D.values(*D.quantize(np64(dY)))
    xt64, dyt64 = D.values(*D.quantize(np64(X).T)), D.values(*D.quantize(np64(dY).T))
    for got, l, r in ((ssg.mm_fp8(X.cuda(), w, ws), x64, w64.T), (ssg.mm_fp8(dY.cuda(), wt, wts), dy64, w64),
                      (ssg.mm_fp8(dyt, xt, xts, xscales=dyts), dyt64, xt64.T)):
        D.check(got, l @ r, np.abs(l) @ np.abs(r), l.shape[1], "linear")


def test_streams_and_workspace():
    X, W = D.randn((300, 500), "bf16", 1).cuda(), D.randn((200, 500), "bf16", 2).cuda()
    w, ws = ssg.fp8_quantize(W, block=128)
    want = ssg.mm_fp8(X, w, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w2, ws2 = ssg.fp8_quantize(W, block=128, stream=s)
    Y = ssg.mm_fp8(X, w2, ws2, stream=s)
    v = ssg.fp8_dequantize(w2, ws2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(Y, want) and torch.equal(v, ssg.fp8_dequantize(w, ws))
    need = ssg.ssg_mm_fp8_workspace_bytes(X, w, ws)
    assert need > 0
    Y = torch.empty_like(want)
    ssg.ssg_mm_fp8(X, w, ws, Y, ws=torch.full((need,), 0x7F, dtype=torch.uint8).cuda())
    assert torch.equal(Y, want)
    with pytest.raises(ssg.SsgError):
        ssg.ssg_mm_fp8(X, w, ws, Y, ws=torch.empty(need - 16, dtype=torch.uint8).cuda())


@pytest.mark.parametrize("N", [3, 200])
def test_graph_replays(N):
    E, M, K = 4, 130, 300
    X = torch.empty(N, K, dtype=torch.bfloat16).cuda()
    W = torch.empty(E, M, K, dtype=torch.bfloat16).cuda()
    offs = torch.empty(E + 1, dtype=torch.int32).cuda()

    def step():
        w, ws = ssg.fp8_quantize(W, block=128)
        Y = ssg.grouped_mm_fp8(X, w, ws, offs, out_dtype=torch.bfloat16)
        xt, xts = ssg.fp8_quantize(X, transpose=True)
        yt, yts = ssg.fp8_quantize(Y, transpose=True)
        return Y, ssg.mm_fp8(yt, xt, xts, xscales=yts), ssg.mm_fp8(X, w[0], ws[0])

    def fill(seed):
        X.copy_(D.randn((N, K), "bf16", seed))
        W.copy_(D.randn((E, M, K), "bf16", seed + 9))
        offs.copy_(torch.tensor([0, 1, 1, N - 1, N - 1 + seed % 2], dtype=torch.int32))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (2, 3, 4):
        fill(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
