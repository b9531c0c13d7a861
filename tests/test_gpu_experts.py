"""Routing, the order of expert rows, gather, combine and their gradients through
the public calls, against 64-bit definitions."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _experts as D
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


# ---------------------------------------------------------------- routing
#
# A weight is expf of a difference (off by a step of 2^-24 of it in the exponent
# and a step of 2^-23 itself), sums of at most E of them, and a division:
# (E + 16 + 2 range) steps of 2^-23, where range is the largest difference of two
# logits of the row that still counts (below 2^-126 of the largest: nothing).

def check_route(l, k, bias=None, **opt):
    lg = l.cuda()
    w, e = ssg.route(lg, k, bias=None if bias is None else bias.cuda(), **opt)
    assert w.dtype == torch.float32 and e.dtype == torch.int32
    l64 = np64(l)
    rw, re = D.route(l64, k, bias=None if bias is None else np64(bias), **opt)
    assert np.array_equal(e.cpu().numpy(), re)
    scale, E = opt.get("scale", 1.0), l.shape[1]
    fin = l64[np.isfinite(l64)]
    span = min(104.0, np.ptp(fin)) if fin.size else 0.0
    bound = (E + 16 + 2 * span) * 2.0 ** -23
    D.close(w, rw, bound * np.abs(rw) + scale * 2.0 ** -120, "weights")
    for renorm in {True, opt.get("renorm", True)}:
        o = dict(score=opt.get("score", "softmax"), renorm=renorm, scale=scale)
        dw = D.randn(w.shape, "f32", 5 * k + E)
        d = ssg.route_backward(dw.cuda(), lg, e, **o)
        assert d.dtype == l.dtype and d.shape == l.shape
        ref, mag = D.route_grad(np64(dw), l64, re, **o)
        D.close(d, ref, 4 * bound * mag + scale * 2.0 ** -120, "dlogits")
    return w, e


# (N, E, k, groups, top_groups): lanes of one and of several experts, groups of
# odd sizes and numbers, as many choices as there are experts
SHAPES = [(1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 8, 2, 1, 1), (64, 64, 6, 8, 3), (33, 60, 4, 5, 2), (70, 96, 8, 6, 3),
          (9, 128, 16, 1, 1), (40, 256, 8, 8, 4), (17, 160, 6, 8, 3), (6, 257, 17, 1, 1), (5, 1000, 64, 40, 9),
          (3, 1024, 10, 1, 1), (4, 1023, 8, 33, 5), (2, 64, 64, 64, 64), (130, 100, 3, 50, 7), (257, 16, 16, 16, 16)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,E,k,groups,top", SHAPES)
def test_route(dt, score, N, E, k, groups, top):
    l = D.randn((N, E), dt, N + E, 2.0)
    bias = D.randn((E,), "f32", E, 0.2)
    for b in (None, bias):
        for gs in ("max", "top2") if groups > 1 else ("max",):
            check_route(l, k, b, score=score, groups=groups, top_groups=top, group_score=gs, renorm=(N + k) % 2 == 0,
                        scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties(score):
    # few different logits: many experts and groups tie, and the lower one wins
    l = torch.randint(-2, 3, (200, 96), generator=torch.Generator().manual_seed(1)).float() * 0.5
    l[::3] *= -0.0                                      # zeros of both signs
    for groups, top in ((1, 1), (8, 3), (6, 4)):
        for gs in ("max", "top2"):
            check_route(l, 7, score=score, groups=groups, top_groups=top, group_score=gs)
            check_route(l, 7, torch.zeros(96), score=score, groups=groups, top_groups=top, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_masks(score, groups, top):
    inf = float("inf")
    l = D.randn((12, 64), "f32", 3)
    l[0] = -inf                                         # a padded token
    l[1, 1:] = -inf                                     # one expert left
    l[2, :60] = -inf                                    # a last few
    l[3, ::2] = -inf
    l[4, 16:] = -inf                                    # groups without experts
    l[5] = torch.finfo(torch.float32).min               # the lowest number is not a mask
    l[6] -= 200.0                                       # every sigmoid underflows
    l[7, 5] = 300.0
    bias = D.randn((64,), "f32", 4, 0.1)
    bias[[3, 17]] = -inf
    for b in (None, bias):
        for gs in ("max", "top2"):
            w, e = check_route(l, 6, b, score=score, groups=groups, top_groups=top, group_score=gs)
            assert (e[0] == -1).all() and (w[0] == 0).all()
            if b is not None:
                assert not ((e == 3) | (e == 17)).any()
    w, e = ssg.route(l.cuda(), 6, score=score)
    total = w.sum(dim=1).cpu()
    assert (total[1:] - 1).abs().max() < 7 * 2.0 ** -23


def test_route_nan_and_infinity():
    nan, inf = float("nan"), float("inf")
    l = D.randn((4, 40), "f32", 9)
    l[1, [7, 30]] = nan
    l[2, 11] = inf
    for score in ("softmax", "sigmoid"):
        w, e = ssg.route(l.cuda(), 3, score=score)
        w, e = w.cpu(), e.cpu()
        assert e[1, :2].tolist() == [7, 30] and torch.isnan(w[1]).all()
        assert e[2, 0] == 11
        assert torch.isfinite(w[[0, 3]]).all()
    w, e = ssg.route(l.cuda(), 3, score="sigmoid", renorm=False)
    assert torch.isnan(w[1, :2]).all() and torch.isfinite(w[1, 2]) and w[2, 0] == 1.0
    for groups, gs in ((4, "max"), (4, "top2")):
        for b in (None, torch.zeros(40).cuda()):
            e = ssg.route(l.cuda(), 3, score="sigmoid", groups=groups, top_groups=2, group_score=gs, bias=b)[1].cpu()
            assert e[1, :2].tolist() == [7, 30] and e[2, 0] == 11


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (5, 3)])
def test_route_far_logits(score, groups, top):
    # where exponentials overflow and underflow, in 32 and in 64 bits, and the type's ends
    far = [0.0, 1e-30, 20.0, 87.0, 89.0, 104.0, 700.0, 709.5, 710.5, 744.0, 746.0, 1999.0, 2001.0, 1e30, 3.4028235e38]
    values = torch.tensor([s * v for v in far for s in (1, -1)])
    g = torch.Generator().manual_seed(6)
    l = values[torch.randint(0, len(values), (200, 40), generator=g)]
    bias = D.randn((40,), "f32", 8)
    opt = dict(score=score, groups=groups, top_groups=top)
    w, e = ssg.route(l.cuda(), 5, bias=bias.cuda(), **opt)
    rw, re = D.route(np64(l), 5, bias=np64(bias), **opt)
    assert np.array_equal(e.cpu().numpy(), re)
    # the weights' bound of the tests above, with differences up to 104 (below: nothing)
    D.close(w, rw, (40 + 16 + 2 * 104) * 2.0 ** -23 * np.abs(rw) + 2.0 ** -120, "weights")
    w, e = ssg.route(l.cuda(), 5, **opt)
    rw, re = D.route(np64(l), 5, **opt)
    assert np.array_equal(e.cpu().numpy(), re)
    D.close(w, rw, (40 + 16 + 2 * 104) * 2.0 ** -23 * np.abs(rw) + 2.0 ** -120, "weights")
    d = ssg.route_backward(torch.ones(200, 5).cuda(), l.cuda(), e, score=score)
    assert torch.isfinite(d).all()


def test_route_strides_and_outputs_in_place():
    wide = D.randn((37, 200), "bf16", 2).cuda()
    l = wide[:, 3:3 + 65]
    w, e = ssg.route(l, 5)
    w2, e2 = ssg.route(l.contiguous(), 5)
    assert torch.equal(w, w2) and torch.equal(e, e2)
    wb, eb = torch.full((37, 9), 7.0).cuda(), torch.full((37, 8), 7, dtype=torch.int32).cuda()
    ssg.ssg_route(l, wb[:, 2:7], eb[:, 1:6])
    assert torch.equal(wb[:, 2:7], w) and torch.equal(eb[:, 1:6], e)
    assert (wb[:, :2] == 7).all() and (wb[:, 7:] == 7).all() and (eb[:, :1] == 7).all() and (eb[:, 6:] == 7).all()
    db = torch.full((37, 80), 7.0, dtype=torch.bfloat16).cuda()
    ssg.ssg_route_backward(wb[:, 2:7], l, eb[:, 1:6], db[:, 4:69])
    assert torch.equal(db[:, 4:69], ssg.route_backward(w, l, e))
    assert (db[:, :4] == 7).all() and (db[:, 69:] == 7).all()


def test_route_gradient_against_differences():
    """The gradient's slope along a direction against a central difference of the
    64-bit formula with the choice held: its error is the third derivative's,
    below 1e-6 for steps of 1e-4 and scores' derivatives below 1."""
    l, dw = D.randn((20, 30), "f32", 6), D.randn((20, 4), "f32", 7)
    d = D.randn((20, 30), "f32", 8).double().numpy()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _, e = ssg.route(l.cuda(), 4, score=score, renorm=renorm)
            got = np64(ssg.route_backward(dw.cuda(), l.cuda(), e, score=score, renorm=renorm))
            at = e.cpu().long().numpy()

            def loss(x):
                s = np.take_along_axis(D.scores(x, score), at, axis=1)
                if renorm:
                    s = s / s.sum(axis=1, keepdims=True)
                return (s * np64(dw)).sum(axis=1)

            h = 1e-4
            slope = (loss(np64(l) + h * d) - loss(np64(l) - h * d)) / (2 * h)
            assert np.abs((got * d).sum(axis=1) - slope).max() < 2e-5


def test_route_gradient_of_other_experts():
    # out of range and masked experts count for nothing, repeated ones add up
    l = D.randn((3, 12), "f32", 1)
    l[2, 4] = -float("inf")
    e = torch.tensor([[3, 12, -1], [5, 5, 2], [4, 1, 2 ** 31 - 1]], dtype=torch.int32)
    dw = D.randn((3, 3), "f32", 2)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = ssg.route_backward(dw.cuda(), l.cuda(), e.cuda(), score=score, renorm=renorm)
            ref, mag = D.route_grad(np64(dw), np64(l), e.numpy(), score=score, renorm=renorm)
            D.close(got, ref, 100 * 2.0 ** -23 * mag, "dlogits")


# ---------------------------------------------------------------- the order

@pytest.mark.parametrize("E", [1, 2, 7, 64, 256, 1000, 1024])
@pytest.mark.parametrize("N,k", [(1, 1), (3, 5), (64, 1), (65, 1), (16, 4), (2048, 4), (4097, 1), (8193, 1), (3001, 6), (50000, 3), (150001, 2)])
def test_order(E, N, k):
    g = np.random.default_rng(E + N)
    e = np.minimum(np.floor(E * g.random((N, k)) ** 2), E - 1).astype(np.int32)
    e[g.random((N, k)) < 0.05] = -1
    offs, rows, pos = ssg.expert_order(torch.from_numpy(e).cuda(), E)
    ro, rr, rp = D.order(e, E)
    assert np.array_equal(offs.cpu().numpy(), ro)
    assert np.array_equal(rows.cpu().numpy(), rr)
    assert np.array_equal(pos.cpu().numpy(), rp)


def test_order_extremes():
    for e, E in ((np.full((100, 3), 5), 6), (np.full((9000, 2), -1), 6), (np.full((9000, 2), 0), 1),
                 (np.array([[2 ** 31 - 1, -2 ** 31, 3, 4]]), 4), (np.zeros((0, 4)), 5), (np.zeros((7, 0)), 5),
                 (np.zeros((2, 2)), 0)):
        e = e.astype(np.int32)
        offs, rows, pos = ssg.expert_order(torch.from_numpy(e).cuda(), E)
        ro, rr, rp = D.order(e, E)
        assert np.array_equal(offs.cpu().numpy(), ro) and np.array_equal(rows.cpu().numpy(), rr)
        assert np.array_equal(pos.cpu().numpy(), rp)


def test_order_strided_and_workspace():
    wide = torch.randint(0, 9, (5000, 7), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    e = wide[:, 2:5]
    want = ssg.expert_order(e.contiguous(), 9)
    for a, b in zip(ssg.expert_order(e, 9), want):
        assert torch.equal(a, b)
    need = ssg.ssg_expert_order_workspace_bytes(5000, 3, 9)
    assert need > 0
    out = [torch.empty_like(t) for t in want]
    ssg.ssg_expert_order(e, 9, *out, ws=torch.full((need,), 255, dtype=torch.uint8).cuda())
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    with pytest.raises(ssg.SsgError):
        ssg.ssg_expert_order(e, 9, *out, ws=torch.empty(need - 1, dtype=torch.uint8).cuda())


# ---------------------------------------------------------------- gather, combine, gradients

def choices(N, k, E, seed, empty=0.1):
    g = np.random.default_rng(seed)
    e = np.stack([g.permutation(max(E, k))[:k] for _ in range(N)]) if N and k else np.zeros((N, k))
    e = np.where(g.random((N, k)) < empty, -1, e % E if E else -1).astype(np.int32)
    return torch.from_numpy(e)


SIZES = [(1, 1, 1), (1, 4, 4096), (5, 2, 7), (16, 8, 100), (70, 3, 264), (33, 6, 1000), (300, 2, 2048), (9, 64, 72),
         (4, 5, 4099)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N,k,C", SIZES)
def test_gather_and_combine(dt, N, k, C):
    e = choices(N, k, 64, N + k + C)
    offs, rows, pos = ssg.expert_order(e.cuda(), 64)
    _, rr, rp = D.order(e.numpy(), 64)
    X = D.randn((N, C), dt, C)
    Y = ssg.expert_gather(X.cuda(), pos, rows)
    want = X[torch.from_numpy(rr.clip(0) // k).long()]
    want[torch.from_numpy(rr < 0)] = 0
    assert torch.equal(Y.cpu(), want)

    Ye = D.randn((N * k, C), dt, C + 1)                 # rows of nobody: numbers that must not count
    Ye[torch.from_numpy(rr < 0)] = float("nan")
    w = D.randn((N, k), "f32", C + 2)
    y64, w64, there = np64(Ye)[rp.clip(0)], np64(w)[:, :, None], (rp >= 0)[:, :, None]
    for weights in (w, None):
        f = w64 if weights is not None else np.ones_like(w64)
        terms = np.where(there, f * y64, 0.0)
        mag = np.abs(terms).sum(axis=1)
        for out in {D.TORCH[dt], torch.float32}:
            O = ssg.expert_combine(Ye.cuda(), pos, None if weights is None else w.cuda(), out_dtype=out)
            assert O.dtype == out
            # k multiply-adds, a rounding each
            D.close(O, terms.sum(axis=1), k * 2.0 ** -24 * mag, "combine")

    dO = D.randn((N, C), dt, C + 3)
    dY, dw = ssg.expert_combine_backward(dO.cuda(), Ye.cuda(), pos, rows, w.cuda())
    assert dY.dtype == D.TORCH[dt] and dw.dtype == torch.float32
    ref = np.zeros((N * k, C))
    src = rr >= 0
    ref[src] = np64(w).reshape(-1)[rr[src]][:, None] * np64(dO)[rr[src] // k]
    D.close(dY, ref, 2.0 ** -24 * np.abs(ref), "dY")    # one rounding in fp32, one to the type
    prod = np.where(there, y64 * np64(dO)[:, None, :], 0.0)
    # C products (inexact for fp32) added in any order
    D.close(dw, prod.sum(axis=2), (C + 8) * 2.0 ** -23 * np.abs(prod).sum(axis=2), "dweights")


def test_rows_strided_and_guarded():
    N, k, C = 21, 4, 130
    e = choices(N, k, 10, 3)
    _, rows, pos = ssg.expert_order(e.cuda(), 10)
    for dt, pad in (("bf16", 3), ("f16", 8), ("f32", 4)):
        T = D.TORCH[dt]
        X = D.randn((N, C + pad + 5), dt, 1).cuda()[:, pad:pad + C]
        Yb = torch.full((N * k, C + 2 * pad), 7.0, dtype=T).cuda()
        Y = Yb[:, pad:pad + C]
        ssg.ssg_expert_gather(X, pos, rows, Y)
        assert torch.equal(Y, ssg.expert_gather(X.contiguous(), pos, rows))
        Ob = torch.full((N, C + 2 * pad), 7.0, dtype=T).cuda()
        w = D.randn((N, k + 3), "f32", 2).cuda()[:, 1:1 + k]
        ssg.ssg_expert_combine(Y, pos, Ob[:, pad:pad + C], w)
        assert torch.equal(Ob[:, pad:pad + C], ssg.expert_combine(Y.contiguous(), pos, w.contiguous()))
        dYb, dwb = torch.full_like(Yb, 7.0), torch.full((N, k + 2), 7.0).cuda()
        ssg.ssg_expert_combine_backward(X, Y, pos, rows, w, dYb[:, pad:pad + C], dwb[:, 1:1 + k])
        dY, dw = ssg.expert_combine_backward(X.contiguous(), Y.contiguous(), pos, rows, w.contiguous())
        assert torch.equal(dYb[:, pad:pad + C], dY)
        # (rows of 16-byte pieces and of elements add the products in another order)
        prod = (X.double()[:, None] * Y.double()[pos.long().clamp_min(0)]).abs().sum(dim=2)
        assert ((dwb[:, 1:1 + k] - dw).abs().double() <= (C + 8) * 2.0 ** -22 * prod + 1e-30).all()
        for b in (Yb, Ob, dYb):
            assert (b[:, :pad] == 7).all() and (b[:, pad + C:] == 7).all()
        assert (dwb[:, 0] == 7).all() and (dwb[:, 1 + k:] == 7).all()


def test_rows_of_a_wrong_order_stay_in_range():
    # entries out of range count as -1; what they leave out is not written
    N, k, C = 6, 3, 24
    pos = torch.arange(N * k, dtype=torch.int32).view(N, k)
    pos[0, 0], pos[2, 1], pos[5, 2] = N * k, -5, 2 ** 31 - 1
    rows = torch.arange(N * k, dtype=torch.int32)
    rows[1], rows[4] = N * k, -2 ** 31
    X = D.randn((N, C), "f16", 1)
    Yb = torch.full((N * k + 2, C), 7.0, dtype=torch.float16).cuda()
    ssg.ssg_expert_gather(X.cuda(), pos.cuda(), rows.cuda(), Yb[1:-1])
    assert (Yb[0] == 7).all() and (Yb[-1] == 7).all()
    w = torch.ones(N, k)
    O = ssg.expert_combine(Yb[1:-1], pos.cuda(), w.cuda())
    assert O.shape == (N, C)
    dYb = torch.full_like(Yb, 7.0)
    dw = torch.empty(N, k).cuda()
    ssg.ssg_expert_combine_backward(X.cuda(), Yb[1:-1], pos.cuda(), rows.cuda(), w.cuda(), dYb[1:-1], dw)
    assert (dYb[0] == 7).all() and (dYb[-1] == 7).all()
    assert dw[0, 0] == 0 and dw[2, 1] == 0 and dw[5, 2] == 0


def test_empty():
    f, i = torch.float16, torch.int32
    w, e = ssg.route(torch.empty(0, 8, dtype=f).cuda(), 2)
    assert w.shape == (0, 2) and e.shape == (0, 2)
    assert ssg.route_backward(w, torch.empty(0, 8, dtype=f).cuda(), e).shape == (0, 8)
    offs, rows, pos = ssg.expert_order(e, 8)
    assert offs.tolist() == [0] * 9 and rows.numel() == 0
    assert ssg.expert_gather(torch.empty(0, 16, dtype=f).cuda(), pos, rows).shape == (0, 16)
    assert ssg.expert_combine(torch.empty(0, 16, dtype=f).cuda(), pos, w).shape == (0, 16)
    none = torch.empty(3, 0, dtype=i).cuda()            # tokens without choices
    O = ssg.expert_combine(torch.empty(0, 16, dtype=f).cuda(), none)
    assert O.shape == (3, 16) and (O == 0).all()
    pos = torch.zeros(2, 1, dtype=i).cuda()             # rows without columns
    dY, dw = ssg.expert_combine_backward(torch.empty(2, 0).cuda(), torch.empty(2, 0).cuda(), pos, pos.view(-1),
                                         torch.ones(2, 1).cuda())
    assert dY.shape == (2, 0) and (dw == 0).all()


# ---------------------------------------------------------------- streams, graphs, a layer

def layer(l, X, W, k, w_out=torch.float32):
    w, e = ssg.route(l, k)
    offs, rows, pos = ssg.expert_order(e, W.shape[0])
    Y = ssg.grouped_mm(ssg.expert_gather(X, pos, rows), W, offs)
    return ssg.expert_combine(Y, pos, w, out_dtype=w_out), e


def test_layer_against_the_formula():
    N, E, k, K, M = 150, 12, 3, 96, 64
    l, X, W = D.randn((N, E), "bf16", 1), D.randn((N, K), "bf16", 2), D.randn((E, M, K), "bf16", 3)
    l[140:] = -float("inf")
    O, e = layer(l.cuda(), X.cuda(), W.cuda(), k)
    w64, e64 = D.route(np64(l), k)
    assert np.array_equal(e.cpu().numpy(), e64)
    ref, tol = np.zeros((N, M)), np.zeros((N, M))
    for n in range(N):
        for j in range(k):
            if e64[n, j] >= 0:
                y, m = np64(X)[n] @ np64(W)[e64[n, j]].T, np.abs(np64(X)[n]) @ np.abs(np64(W)[e64[n, j]]).T
                ref[n] += w64[n, j] * y
                # the product's sum and its rounding to bf16, and the weight's
                t = (K + 16) * 2.0 ** -23 * m
                tol[n] += w64[n, j] * (t + (np.abs(y) + t) * 2.0 ** -8 + 60 * 2.0 ** -23 * np.abs(y))
    D.close(O, ref, tol + k * 2.0 ** -23 * np.abs(ref), "layer")
    assert (O[140:] == 0).all()


def test_streams():
    l, X, W = D.randn((90, 8), "f16", 1).cuda(), D.randn((90, 64), "f16", 2).cuda(), D.randn((8, 32, 64), "f16", 3).cuda()
    want = layer(l, X, W, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(l, X, W, 2)
    w, e = ssg.route(l, 2, stream=s)
    offs, rows, pos = ssg.expert_order(e, 8, stream=s)
    Xs = ssg.expert_gather(X, pos, rows, stream=s)
    O = ssg.expert_combine(ssg.grouped_mm(Xs, W, offs, stream=s), pos, w, out_dtype=torch.float32, stream=s)
    d = ssg.route_backward(w, l, e, stream=s)
    dY, dw = ssg.expert_combine_backward(X, Xs, pos, rows, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(O, want[0]) and torch.equal(e, want[1])
    assert torch.equal(d, ssg.route_backward(w, l, e))
    for a, b in zip((dY, dw), ssg.expert_combine_backward(X, Xs, pos, rows, w)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N", [40, 6000])               # one and several parts of the order
def test_graph_replays(N):
    E, k, K, M = 8, 2, 64, 48
    l, X = torch.empty(N, E, dtype=torch.bfloat16).cuda(), torch.empty(N, K, dtype=torch.bfloat16).cuda()
    W = D.randn((E, M, K), "bf16", 3).cuda()

    def step():
        w, e = ssg.route(l, k, score="sigmoid", bias=torch.zeros(E, device="cuda"))
        offs, rows, pos = ssg.expert_order(e, E)
        Xs = ssg.expert_gather(X, pos, rows)
        O = ssg.expert_combine(ssg.grouped_mm(Xs, W, offs), pos, w)
        dY, dw = ssg.expert_combine_backward(O, ssg.grouped_mm(Xs, W, offs), pos, rows, w)
        return O, dY, ssg.route_backward(dw, l, e, score="sigmoid"), offs

    def fill(seed):
        l.copy_(D.randn((N, E), "bf16", seed))
        l[N - seed:] = -float("inf")
        X.copy_(D.randn((N, K), "bf16", seed + 50))

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
