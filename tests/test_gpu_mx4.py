"""The mx4 format and the products of mx4 weights through the public calls,
against 64-bit definitions."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- the format

@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,K", [(1, 1), (3, 31), (5, 32), (4, 33), (7, 100), (2, 4096), (129, 264), (1000, 96)])
def test_quantize_and_back(dt, R, K):
    a = D.randn((R, K), dt, R + K) * torch.exp2(torch.randint(-9, 9, (R, 1))).to(D.TORCH[dt])
    e, s = ssg.mx4_quantize(a.cuda())
    re, rs = D.mx4_quantize(a.double().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(e.cpu().numpy(), re)
    v = D.mx4_values(re, rs, K)
    for out in ("f16", "bf16", "f32"):
        got = ssg.mx4_dequantize(e, s, K, dtype=D.TORCH[out])
        want = torch.from_numpy(v).to(D.TORCH[out])     # every value is exact in fp32: one rounding
        assert torch.equal(got.cpu(), want), out


def test_quantize_every_tie_and_border():
    # a block per quotient: the borders between codes, their neighbours, both signs
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0]
    rows = []
    for m in mids:
        for d in (0.0, 2.0 ** -10, -(2.0 ** -10)):
            for sgn in (1.0, -1.0):
                rows.append([4.0] + [sgn * (m + d)] * 31)
    a = torch.tensor(rows, dtype=torch.float32)
    for scale in (1.0, 2.0 ** -100, 2.0 ** 100):
        x = a * scale
        e, s = ssg.mx4_quantize(x.cuda())
        re, rs = D.mx4_quantize(x.double().numpy())
        assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(e.cpu().numpy(), re)


def test_quantize_extremes():
    t = torch.finfo(torch.float32)
    inf, nan = float("inf"), float("nan")
    a = torch.zeros(10, 64)
    a[1, 3], a[1, 40] = t.max, -t.max
    a[2, 0], a[2, 33] = t.smallest_normal, t.smallest_normal * 5
    a[3, 1], a[3, 32] = 1e-45, 3e-45                     # subnormal fp32
    a[4, 2], a[4, 3] = inf, 1.0
    a[5, 2], a[5, 3] = -inf, t.max
    a[6, 5], a[6, 6] = nan, 2.0
    a[7, 5], a[7, 6] = nan, inf
    a[8, :] = -0.0
    a[9, 0], a[9, 1] = 2.0 ** -126, 2.0 ** -149
    e, s = ssg.mx4_quantize(a.cuda())
    re, rs = D.mx4_quantize(a.double().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(e.cpu().numpy(), re)
    back = ssg.mx4_dequantize(e, s, 64).cpu()
    assert back[4, 2] == inf and back[4, 3] == 0 and back[5, 2] == -inf
    assert torch.isnan(back[6, :32]).all() and torch.isnan(back[7, :32]).all() and (back[6, 32:] == 0).all()
    f16 = ssg.mx4_dequantize(e, s, 64, dtype=torch.float16).cpu()
    assert f16[1, 3] == inf and f16[3, 1] == 0


def test_quantize_strided_and_unaligned():
    wide = D.randn((40, 301), "bf16", 5).cuda()
    a = wide[:, 7:7 + 130]
    e, s = ssg.mx4_quantize(a)
    re, rs = D.mx4_quantize(a.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(e.cpu().numpy(), re)
    ebuf, sbuf = torch.zeros(40, 95, dtype=torch.uint8).cuda(), torch.zeros(40, 11, dtype=torch.uint8).cuda()
    ssg.ssg_mx4_quantize(a, ebuf[:, 3:83], sbuf[:, 1:6])
    assert torch.equal(ebuf[:, 3:83], e) and torch.equal(sbuf[:, 1:6], s)
    assert (ebuf[:, :3] == 0).all() and (ebuf[:, 83:] == 0).all() and (sbuf[:, 6:] == 0).all()
    out = torch.full((40, 150), 7.0, dtype=torch.float16).cuda()
    ssg.ssg_mx4_dequantize(ebuf[:, 3:83], sbuf[:, 1:6], out[:, 5:135])
    assert torch.equal(out[:, 5:135].double().cpu(), torch.from_numpy(D.mx4_values(re, rs, 130)))
    assert (out[:, :5] == 7).all() and (out[:, 135:] == 7).all()


def test_quantize_stack_and_empty():
    a = D.randn((3, 5, 70), "f16", 9)
    e, s = ssg.mx4_quantize(a.cuda())
    assert e.shape == (3, 5, 48) and s.shape == (3, 5, 3)
    for i in range(3):
        ei, si = ssg.mx4_quantize(a[i].cuda())
        assert torch.equal(e[i], ei) and torch.equal(s[i], si)
    assert ssg.mx4_dequantize(e, s, 70).shape == (3, 5, 70)
    e, s = ssg.mx4_quantize(torch.empty(0, 64, dtype=torch.float16).cuda())
    assert e.shape == (0, 32) and s.shape == (0, 2)


# ---------------------------------------------------------------- products

# (M, K, N): one of everything; decode; around the kernels' borders of 16, 32, 64, 128, 256 rows; odd lengths
SHAPES = [(1, 1, 1), (16, 32, 1), (33, 100, 3), (130, 4096, 1), (300, 1000, 16), (64, 512, 17), (96, 516, 32),
          (257, 160, 33), (260, 333, 65), (500, 1024, 100), (513, 264, 257), (40, 2112, 300), (129, 31, 600)]


def activations(x, N, K, seed):
    """(arguments, float64 values) of activations of type x."""
    if x == "mx4":
        e, s = D.random_mx4((N, K), seed, 120, 130)
        return dict(X=dev(e), xscales=dev(s)), D.mx4_values(e, s, K)
    a = D.randn((N, K), x, seed)
    return dict(X=a.cuda()), a.double().numpy()


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_mm_mx4(x, M, K, N):
    ax, xv = activations(x, N, K, M + K)
    e, s = D.random_mx4((M, K), N + K)
    wv = D.mx4_values(e, s, K)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for out in ["f32", "f16", "bf16"] if x == "mx4" else ["f32", x]:
        Y = ssg.mm_mx4(ax["X"], dev(e), dev(s), xscales=ax.get("xscales"), out_dtype=D.TORCH[out])
        assert Y.dtype == D.TORCH[out]
        D.check(Y, ref, mag, K, "mm_mx4 %s -> %s" % (x, out))


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("N", [2, 40, 300])
def test_mm_mx4_any_scale(x, N):
    # every scale byte a weight can have, blocks of one magnitude next to each
    # other: past fp16's range on both sides, subnormal, and near fp32's top
    M, K = 70, 416
    ax, xv = activations(x, N, K, 3)
    e, s = D.random_mx4((M, K), 4, 118, 124)
    g = np.random.default_rng(5)
    s[1] = g.integers(100, 150, s.shape[1])
    s[17] = g.integers(140, 180, s.shape[1])
    s[20] = g.integers(60, 100, s.shape[1])
    s[40, 3], s[41, 5], s[69, 12], s[2, :] = 0, 1, 0, 0
    wv = D.mx4_values(e, s, K)
    with np.errstate(over="ignore"):
        ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    Y = ssg.mm_mx4(ax["X"], dev(e), dev(s), xscales=ax.get("xscales"))
    # subnormal products may be lost by the matrix unit: a half step of fp32's smallest normal each
    D.check(Y, ref, mag + 2.0 ** -126 * 2.0 ** 23, K, "mm_mx4 scales %s" % x)


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("N", [3, 100])
def test_mm_mx4_nan_scale_and_infinite_activations(x, N):
    M, K = 50, 256
    ax, xv = activations(x, N, K, 7)
    e, s = D.random_mx4((M, K), 8)
    s[33, 2] = 255
    Y = ssg.mm_mx4(ax["X"], dev(e), dev(s), xscales=ax.get("xscales")).cpu()
    assert torch.isnan(Y[:, 33]).all()
    assert torch.isfinite(Y[:, :33]).all() and torch.isfinite(Y[:, 34:]).all()
    if x != "mx4":
        s[33, 2] = 120
        e[:, 5] = 0x22                                   # elements 10 and 11 of every row: 1.0
        X = ax["X"].clone()
        X[1, 10] = float("inf")
        Y = ssg.mm_mx4(X, dev(e), dev(s)).cpu()
        assert (Y[1] == float("inf")).all() and torch.isfinite(Y[0]).all() and torch.isfinite(Y[2:]).all()


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("N", [5, 70])
def test_mm_mx4_strides_and_alignment(x, N):
    M, K = 200, 1056
    nb = K // 32
    e, s = D.random_mx4((M, K), 21)
    wv = D.mx4_values(e, s, K)
    We = torch.full((M, nb * 16 + 37), 0xFF, dtype=torch.uint8).cuda()
    Ws = torch.full((M, nb + 6), 255, dtype=torch.uint8).cuda()
    We[:, 5:5 + nb * 16] = dev(e)
    Ws[:, 3:3 + nb] = dev(s)
    ax, xv = activations(x, N, K, 22)
    X, kw = ax["X"], {}
    Xb = torch.full((N, X.shape[1] + 11), 0x7F if x == "mx4" else float("nan"), dtype=X.dtype).cuda()
    Xb[:, 3:3 + X.shape[1]] = X
    if x == "mx4":
        Xs = torch.full((N, nb + 5), 255, dtype=torch.uint8).cuda()
        Xs[:, 1:1 + nb] = ax["xscales"]
        kw["xscales"] = Xs[:, 1:1 + nb]
    Y = torch.full((N, M + 9), 7.0).cuda()
    ssg.ssg_mm_mx4(Xb[:, 3:3 + X.shape[1]], We[:, 5:5 + nb * 16], Ws[:, 3:3 + nb], Y[:, 4:4 + M], **kw)
    D.check(Y[:, 4:4 + M], xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K, "strided")
    assert (Y[:, :4] == 7).all() and (Y[:, 4 + M:] == 7).all()


def test_mm_mx4_empty():
    e, s = D.random_mx4((40, 64), 1)
    Y = ssg.mm_mx4(torch.empty(0, 64, dtype=torch.bfloat16).cuda(), dev(e), dev(s))
    assert Y.shape == (0, 40)
    Y = ssg.mm_mx4(torch.empty(5, 0, dtype=torch.bfloat16).cuda(), torch.empty(40, 0, dtype=torch.uint8).cuda(),
                   torch.empty(40, 0, dtype=torch.uint8).cuda())
    assert Y.shape == (5, 40) and (Y == 0).all()


# ---------------------------------------------------------------- experts

SIZES = [[1], [0, 1], [3, 0, 5, 1], [16, 17, 15, 0, 1], [40, 33, 0, 64, 7], [200, 0, 0, 130, 1, 64], [1] * 70,
         [300, 90], [5] * 13]


@pytest.mark.parametrize("x", ["f16", "bf16", "mx4"])
@pytest.mark.parametrize("which", range(len(SIZES)))
def test_grouped_mm_mx4(x, which):
    sizes = SIZES[which]
    E, N = len(sizes), sum(sizes)
    M, K = [(100, 200), (33, 512), (260, 96), (64, 1000)][which % 4]
    ax, xv = activations(x, N, K, which)
    e, s = D.random_mx4((E, M, K), which + 50)
    offs = D.offsets(sizes)
    ref, mag = D.grouped(xv, D.mx4_values(e, s, K), offs)
    for out in ("f32", "bf16") if x == "mx4" else ("f32", x):
        Y = ssg.grouped_mm_mx4(ax["X"], dev(e), dev(s), offs.cuda(), xscales=ax.get("xscales"), out_dtype=D.TORCH[out])
        D.check(Y, ref, mag, K, "grouped_mm_mx4 %s -> %s" % (x, out))


@pytest.mark.parametrize("x", ["f16", "mx4"])
@pytest.mark.parametrize("rows", [1, 30])
def test_grouped_mm_mx4_rows_of_no_expert_are_zero(x, rows):
    M, K, sizes = 70, 128, [rows, 0, 2 * rows]
    N = 3 * rows + 50
    ax, xv = activations(x, N, K, 3)
    e, s = D.random_mx4((3, M, K), 4)
    offs = D.offsets(sizes, first=20)
    Y = ssg.grouped_mm_mx4(ax["X"], dev(e), dev(s), offs.cuda(), xscales=ax.get("xscales"))
    ref, mag = D.grouped(xv, D.mx4_values(e, s, K), offs)
    D.check(Y, ref, mag, K, "uncovered rows")
    assert (Y[:20] == 0).all() and (Y[20 + 3 * rows:] == 0).all()


def test_quantized_layer_against_its_16_bit_weights():
    # quantise, multiply, and compare with the product of the dequantised weights
    W = D.randn((4, 300, 512), "bf16", 1, 0.05).cuda()
    X = D.randn((90, 512), "bf16", 2).cuda()
    offs = D.offsets([20, 0, 50, 20])
    e, s = ssg.mx4_quantize(W)
    Wd = ssg.mx4_dequantize(e, s, 512, dtype=torch.bfloat16)
    ref, mag = D.grouped(X.double().cpu().numpy(), Wd.double().cpu().numpy(), offs)
    D.check(ssg.grouped_mm_mx4(X, e, s, offs.cuda()), ref, mag, 512, "mx4")
    D.check(ssg.grouped_mm(X, Wd, offs.cuda(), out_dtype=torch.float32), ref, mag, 512, "16-bit")
    xe, xs = ssg.mx4_quantize(X)
    Xd = ssg.mx4_dequantize(xe, xs, 512).double().cpu().numpy()
    ref, mag = D.grouped(Xd, Wd.double().cpu().numpy(), offs)
    D.check(ssg.grouped_mm_mx4(xe, e, s, offs.cuda(), xscales=xs), ref, mag, 512, "mx4 x mx4")


def test_same_bits_each_call_and_on_another_stream():
    e, s = D.random_mx4((520, 1000), 1)
    for x, N in [("bf16", 7), ("bf16", 90), ("mx4", 300)]:
        ax, _ = activations(x, N, 1000, N)
        We, Ws = dev(e), dev(s)
        Y = ssg.mm_mx4(ax["X"], We, Ws, xscales=ax.get("xscales"))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(3):
            Z = ssg.mm_mx4(ax["X"], We, Ws, xscales=ax.get("xscales"), stream=side)
            side.synchronize()
            assert torch.equal(Y, Z)
