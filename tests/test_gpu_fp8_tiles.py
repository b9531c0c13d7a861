"""The 8-bit products of many rows: operands in every layout that the tiles read or have
copied, long contractions, and the few-row kernels that round their activations.  The
sizes are checked to take the kernel they are meant for, here and without a GPU."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _fp8 as D
from tests import _mm

F8 = torch.float8_e4m3fn


def np64(t):
    return t.detach().cpu().double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(got, xv, wv, what):
    """Against the product of float64 values, on the GPU in 64 bits."""
    x, w = torch.from_numpy(xv).cuda(), torch.from_numpy(wv).cuda()
    ref, mag = np64(x @ w.t()), np64(x.abs() @ w.abs().t())
    if got.dtype == torch.float16:                       # past its range: infinities (65520 rounds to one)
        far = np.abs(ref) > 65520 + (xv.shape[1] + 100) * 2.0 ** -23 * mag
        near = ~far & (np.abs(ref) > 65504)              # or, with the sums' bound, the last number
        g = np64(got)
        assert np.array_equal(g[far], np.copysign(np.inf, ref[far])) and (np.abs(g[near]) >= 65472).all()
        got = torch.from_numpy(np.where(far | near, 0, g)).half()
        ref, mag = np.where(far | near, 0, ref), np.where(far | near, 0, mag)
    D.check(got, ref, mag, xv.shape[1], what)


# ---------------------------------------------------------------- which kernel

# activations, output, M, K, N, experts, rows to a scale of W, tile (0: few rows)
MEANT = [(x, out, M, K, N, 0, block, 128) for x in ("bf16", "e4m3") for out in ("bf16", "f32") for block in (1, 128)
         for M, K in ((260, 700), (260, 701), (150, 384), (140, 256)) for N in (700, 2100)]
MEANT += [("e4m3", "f32", 900, 700, 600, 0, 1, 128), ("e4m3", "f32", 1300, 2100, 700, 0, 1, 128)]
LONG = [(4090, 1300, 4090, 0), (4100, 1300, 4300, 0), (4100, 1300, 5400, 0), (4090, 1152, 4090, 0), (4100, 100, 4090, 0),
        (4100, 128, 4090, 0), (2050, 1300, 4500, 4)]
MEANT += [("e4m3", "bf16", M, K, N, E, 128, 256) for M, K, N, E in LONG]
MEANT += [("e4m3", "bf16", 300, 1300, 1510, 3, b, 128) for b in (1, 128)]
MEANT += [("e4m3", "f32", 300, 1300, 1510, 3, b, 128) for b in (1, 128)]
ROUND = [(x, M, K, N, block) for x in ("bf16", "f16") for M, K, N, block in
         ((600, 2000, 16, 128), (8190, 300, 5, 128), (8190, 2048, 16, 128), (600, 2000, 16, 1), (4090, 131, 1, 1))]


@pytest.mark.parametrize("x,out,M,K,N,E,block,tile", MEANT)
def test_sizes_take_tiles(x, out, M, K, N, E, block, tile):
    dt = {"e4m3": F8, **D.TORCH}
    kernel = ssg.ssg_mm_fp8_select_kernel(dt[x], dt[out], M, N, K, E, block)
    assert kernel[0] == "tiles" and kernel[1] == tile


@pytest.mark.parametrize("x,M,K,N,block", ROUND)
def test_sizes_round_in_the_kernel(x, M, K, N, block):
    kernel = ssg.ssg_mm_fp8_select_kernel(D.TORCH[x], D.TORCH[x], M, N, K, 0, block)
    assert kernel[0] == "few" and kernel[1] == (32 if M > 8000 else 16) and kernel[2] == 16
    assert N * D.blocks(K) * 128 <= 32768


# ---------------------------------------------------------------- layouts

@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K", [700, 701])
@pytest.mark.parametrize("N", [700, 2100])
def test_layouts_give_the_same(N, K, out):
    """Rounded in the call or before it, scales by rows or by blocks, rows at 16 bytes, at
    4 or anywhere: the same bits."""
    out = D.TORCH[out]
    X, W = D.randn((N, K), "bf16", 1).cuda(), D.randn((260, K), "bf16", 2).cuda()
    x, xs = ssg.fp8_quantize(X)
    for block in (128, 1):
        w, ws = ssg.fp8_quantize(W, block=block)
        want = ssg.mm_fp8(X, w, ws, out_dtype=out)
        for a, s in ((x, xs), (x, xs.contiguous()), (x.contiguous(), xs), (x.contiguous(), xs.contiguous())):
            for b, t in ((w, ws), (w.contiguous(), ws.contiguous()), (w, ws.t().contiguous().t())):
                assert torch.equal(ssg.mm_fp8(a, b, t, xscales=s, out_dtype=out), want)
        check(want, D.values(*D.quantize(np64(X))), D.values(*D.quantize(np64(W), block)), "mm_fp8")


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [700, 2100])
def test_strided_unaligned_and_guarded(N, out):
    M, K = 150, 384
    cx, sx = D.random_fp8(N, K, 1)
    for block in (128, 1):
        cw, sw = D.random_fp8(M, K, 2, block)
        xv, wv = D.values(cx, sx.astype(np.float64)), D.values(cw, sw.astype(np.float64))
        for pad in (1, 2, 4, 16):                        # NaN around every operand
            xb = torch.full((N, K + 2 * pad), 0x7F, dtype=torch.uint8).cuda()
            wb = torch.full((M, K + 2 * pad), 0x7F, dtype=torch.uint8).cuda()
            xb[:, pad:pad + K], wb[:, pad:pad + K] = dev(cx), dev(cw)
            sb, tb = torch.full((N, 9), float("nan")).cuda(), torch.full((sw.shape[0] + 2, 5), float("nan")).cuda()
            sb[:, 2:5], tb[1:-1, 1:4] = dev(sx), dev(sw)
            Yb = torch.full((N + 2, M + 6), 7.0, dtype=D.TORCH[out]).cuda()
            ssg.ssg_mm_fp8(xb.view(F8)[:, pad:pad + K], wb.view(F8)[:, pad:pad + K], tb[1:-1, 1:4], Yb[1:-1, 3:3 + M],
                           xscales=sb[:, 2:5])
            check(Yb[1:-1, 3:3 + M], xv, wv, "mm_fp8")
            assert (Yb[:, :3] == 7).all() and (Yb[:, 3 + M:] == 7).all() and (Yb[0] == 7).all() and (Yb[-1] == 7).all()
        for K2 in (383, 381, 260, 129):                  # the rest of a row is not read into the sums
            xb, wb, nb = dev(cx), dev(cw), D.blocks(K2)
            xb[:, K2:], wb[:, K2:] = 0x7F, 0x7F
            Y = ssg.mm_fp8(xb.view(F8)[:, :K2], wb.view(F8)[:, :K2], dev(sw)[:, :nb], xscales=dev(sx)[:, :nb],
                           out_dtype=D.TORCH[out])
            check(Y, D.values(cx[:, :K2], sx[:, :nb].astype(np.float64)), D.values(cw[:, :K2], sw[:, :nb].astype(np.float64)),
                  "mm_fp8")


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("N", [700, 2100])
def test_nan_and_infinity_stay_in_their_rows(N, block, out):
    X, W, out = D.randn((N, 256), "bf16", 1), D.randn((140, 256), "bf16", 2), D.TORCH[out]
    w, ws = ssg.fp8_quantize(W.cuda(), block=block)
    want = ssg.mm_fp8(X.cuda(), w, ws, out_dtype=out)
    X[1, 7], X[3, 200], X[N - 1, 255] = float("nan"), float("inf"), float("nan")
    Y = ssg.mm_fp8(X.cuda(), w, ws, out_dtype=out)
    bad = [1, 3, N - 1]
    assert torch.isnan(Y[bad]).all()
    keep = [n for n in range(N) if n not in bad]
    assert torch.equal(Y[keep], want[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("N,M,K", [(700, 600, 900), (2100, 700, 1300)])
def test_a_weight_gradient_reads_scales_as_they_are_quantised(N, M, K):
    X, dY = D.randn((N, K), "bf16", 1), D.randn((N, M), "bf16", 3)
    xt, xts = ssg.fp8_quantize(X.cuda(), transpose=True)
    dyt, dyts = ssg.fp8_quantize(dY.cuda(), transpose=True)
    assert xts.stride(0) == 1 and dyts.stride(0) == 1       # neighbours: nothing is rearranged
    got = ssg.mm_fp8(dyt, xt, xts, xscales=dyts)
    check(got, D.values(*D.quantize(np64(dY).T)), D.values(*D.quantize(np64(X).T)), "dW")
    assert torch.equal(ssg.mm_fp8(dyt, xt, xts.contiguous(), xscales=dyts.contiguous()), got)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [700, 2100])
def test_workspace(N, out):
    X, W, out = D.randn((N, 384), "bf16", 1).cuda(), D.randn((150, 384), "bf16", 2).cuda(), D.TORCH[out]
    w, ws = ssg.fp8_quantize(W, block=128)
    want = ssg.mm_fp8(X, w, ws, out_dtype=out)
    need = ssg.ssg_mm_fp8_workspace_bytes(X, w, ws, out_dtype=out)
    assert need > 0
    Y = torch.empty_like(want)
    ssg.ssg_mm_fp8(X, w, ws, Y, ws=torch.full((need,), 0x7F, dtype=torch.uint8).cuda())
    assert torch.equal(Y, want)
    with pytest.raises(ssg.SsgError):
        ssg.ssg_mm_fp8(X, w, ws, Y, ws=torch.empty(need - 16, dtype=torch.uint8).cuda())


# ---------------------------------------------------------------- long contractions, experts

@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,E", LONG)
def test_large_tiles(M, K, N, E, out):
    """More blocks than LDS has places, whole and ending inside one; tiles as they are and
    cut in two and in four."""
    g = np.random.default_rng(M + K + N)
    cx, sx = D.random_fp8(N, K, 1)
    sx, mats = sx * np.float32(2.0 ** -9), max(E, 1)
    xv = D.values(cx, sx.astype(np.float64))
    w = [D.random_fp8(M, K, 2 + e, 128) for e in range(mats)]
    Yb = torch.full((N + 1, M + 3), 7.0, dtype=D.TORCH[out]).cuda()
    view, X, xs = Yb[:N, :M], D.elements(cx), dev(sx)
    offs = [0, N] if not E else [0, *sorted(int(v) for v in g.integers(0, N, E - 1)), N - 5]
    if E:
        offs = sorted(offs)
        ssg.ssg_grouped_mm_fp8(X, D.elements(np.stack([c for c, _ in w])), dev(np.stack([s for _, s in w])),
                               torch.tensor(offs, dtype=torch.int32).cuda(), view, xscales=xs)
    else:
        ssg.ssg_mm_fp8(X, D.elements(w[0][0]), dev(w[0][1]), view, xscales=xs)
    for e, (a, b) in enumerate(zip(offs[:-1], offs[1:])):
        if b > a:
            check(Yb[a:b, :M], xv[a:b], D.values(w[e][0], w[e][1].astype(np.float64)), "expert %d" % e)
    assert (Yb[offs[-1]:N, :M] == 0).all() and (Yb[N] == 7).all() and (Yb[:, M:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pad", [0, 1])
def test_experts_in_every_layout(block, pad, out):
    E, M, K, sizes = 3, 300, 1300, [800, 0, 700]
    offs = _mm.offsets(sizes, 4)
    N = 4 + sum(sizes) + 6
    X, W = D.randn((N, K), "bf16", 1), D.randn((E, M, K), "bf16", 2, 0.05)
    x, xs = ssg.fp8_quantize(X.cuda())
    w, ws = ssg.fp8_quantize(W.cuda(), block=block)
    if pad:                                              # rows that begin anywhere, scales that are no neighbours
        wide = torch.full((E, M, K + 3), 0x7F, dtype=torch.uint8).cuda().view(F8)
        wide[..., 1:1 + K] = w
        w, ws, x, xs = wide[..., 1:1 + K], ws.contiguous(), x.contiguous(), xs.contiguous()
    Y = ssg.grouped_mm_fp8(x, w, ws, offs.cuda(), xscales=xs, out_dtype=D.TORCH[out])
    xv = D.values(*D.quantize(np64(X)))
    for e, a, b in _mm.segments(offs.tolist(), N):
        if b > a:
            check(Y[a:b], xv[a:b], D.values(*D.quantize(np64(W)[e], block)), "expert %d" % e)
    assert (Y[:4] == 0).all() and (Y[N - 6:] == 0).all()
    assert torch.equal(ssg.grouped_mm_fp8(X.cuda(), w, ws, offs.cuda(), out_dtype=D.TORCH[out]), Y)


# ---------------------------------------------------------------- activations rounded in the kernel

@pytest.mark.gpu
@pytest.mark.parametrize("x,M,K,N,block", ROUND)
def test_rounding_in_the_kernel(x, M, K, N, block):
    X = D.randn((N, K), x, 1)
    c, s = D.random_fp8(M, K, 2, block)
    s = s * np.float32(2.0 ** -8)
    got = ssg.mm_fp8(X.cuda(), D.elements(c), dev(s), out_dtype=D.TORCH[x])
    check(got, D.values(*D.quantize(np64(X))), D.values(c, s.astype(np.float64)), "mm_fp8")


# ---------------------------------------------------------------- graphs and streams

def steps():
    """(inputs, function) of products by every tile: 256 x 256, cut, 128 x 128, split."""
    X, W = torch.empty(4100, 300, dtype=torch.bfloat16).cuda(), torch.empty(4100, 300, dtype=torch.bfloat16).cuda()
    x, w = torch.empty(599, 2000, dtype=torch.bfloat16).cuda(), torch.empty(250, 2000, dtype=torch.bfloat16).cuda()

    def run():
        e, s = ssg.fp8_quantize(W, block=128)
        f, t = ssg.fp8_quantize(w, block=128)
        big = ssg.mm_fp8(X, e, s, out_dtype=torch.bfloat16)
        xt, xts = ssg.fp8_quantize(x, transpose=True)
        return (big, ssg.mm_fp8(X[:2100], e, s), ssg.mm_fp8(x, f, t, out_dtype=torch.float16),
                ssg.mm_fp8(x, f, t), ssg.mm_fp8(xt, xt, xts, xscales=xts))

    def fill(seed):
        for i, a in enumerate((X, W, x, w)):
            a.copy_(D.randn(tuple(a.shape), "bf16", seed + 10 * i, 0.25))
    return run, fill


def test_the_steps_take_these_kernels():
    k, b = ssg.ssg_mm_fp8_select_kernel, torch.bfloat16
    assert k(b, b, 4100, 4100, 300)[1] == 256 and k(b, torch.float32, 4100, 2100, 300)[1] == 128
    assert k(b, torch.float16, 250, 599, 2000)[3] > 1 and k(b, torch.float32, 250, 599, 2000)[3] > 1
    assert k(F8, torch.float32, 2000, 2000, 599, 0, 1)[0] == "tiles"


@pytest.mark.gpu
def test_graph_replays():
    run, fill = steps()
    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (2, 3, 4):
        fill(seed)
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_streams_at_once():
    run, fill = steps()
    fill(5)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(out, want):
            assert torch.equal(a, b)
