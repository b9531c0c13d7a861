"""Every kernel that the choice between them can make, against 64-bit products:
few rows and tiles, each size of workgroup, whole and split contractions, for
every operator and operand type."""
import math
import random

import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _mm as D

# (M, N, K, E) by operator and by what the activations hold (16-bit, mx4): the
# smallest of many random products that take each kernel
CASES = {
    ("grouped_mm", "16"): [
        (18, 3, 80, 2), (18, 20, 8629, 2), (209, 307, 78, 2), (22, 250, 13616, 2), (374, 365, 71, 3),
        (78, 186, 11214, 2), (409, 664, 73, 5), (293, 227, 11577, 2), (19, 488, 77, 2), (21, 331, 1124, 2),
        (307, 6522, 76, 12), (27, 2410, 2067, 3), (133, 7561, 79, 22)],
    ("grouped_mm_dw", "16"): [
        (1, 89, 19, 2), (215, 71, 18, 82), (141, 87, 132, 48)],
    ("grouped_mm_dx", "16"): [
        (70, 7, 18, 2), (1086, 6, 18, 2), (73, 7535, 270, 10), (2020, 2329, 20, 7), (71, 7982, 135, 16)],
    ("grouped_mm_mx4", "16"): [
        (19, 2, 75, 2), (18, 8, 13991, 2), (39, 2208, 72, 16), (35, 300, 21767, 2), (218, 318, 108, 2),
        (73, 93, 11160, 2), (463, 316, 72, 2), (72, 180, 14397, 3), (315, 458, 4009, 3), (40, 338, 64917, 3),
        (2118, 94, 3142, 2), (101, 436, 27500, 5), (639, 416, 3241, 3), (215, 297, 25306, 2), (22, 420, 74, 2),
        (21, 430, 1209, 2), (280, 6268, 86, 14), (25, 2402, 2171, 6), (312, 6495, 70, 2)],
    ("grouped_mm_mx4", "mx4"): [
        (18, 2, 96, 2), (18, 12, 15264, 2), (39, 1549, 96, 57), (37, 276, 24992, 2), (193, 306, 96, 2),
        (73, 251, 12960, 2), (198, 556, 96, 4), (51, 256, 33568, 2), (35, 3477, 2784, 34), (40, 404, 60256, 9),
        (50, 3783, 3616, 25), (947, 274, 2272, 2), (173, 196, 63392, 2), (30, 385, 96, 2), (62, 364, 4192, 2),
        (281, 6364, 96, 12), (25, 5695, 4256, 4), (797, 2306, 96, 2)],
    ("mm_mx4", "16"): [
        (18, 3, 73, 1), (19, 6, 11925, 1), (810, 151, 82, 1), (458, 133, 72, 1), (55, 146, 11381, 1),
        (900, 143, 77, 1), (131, 119, 12927, 1), (1141, 124, 3402, 1), (97, 147, 63644, 1), (1484, 156, 3985, 1),
        (440, 141, 42735, 1), (1794, 149, 2852, 1), (193, 152, 58168, 1), (18, 184, 72, 1), (26, 166, 1004, 1),
        (525, 6173, 79, 1), (19, 5037, 1091, 1), (280, 6260, 71, 1)],
    ("mm_mx4", "mx4"): [
        (18, 2, 96, 1), (18, 6, 14560, 1), (1354, 94, 8736, 1), (437, 151, 96, 1), (67, 97, 17504, 1),
        (915, 130, 96, 1), (114, 138, 28384, 1), (8295, 2, 2656, 1), (1028, 4, 57952, 1), (1774, 136, 3424, 1),
        (1702, 159, 2528, 1), (312, 110, 64352, 1), (18, 170, 96, 1), (19, 165, 3616, 1), (605, 5428, 96, 1),
        (22, 5264, 4384, 1), (287, 5631, 96, 1)],
}
# contractions of many stages in the largest tiles, their halves and quarters; a
# decode batch of a large weight, and one spread over many experts
CASES["grouped_mm", "16"] += [(1290, 2200, 1058, 2)]
CASES["grouped_mm_dx", "16"] += [(1058, 2200, 1290, 2), (700, 4100, 2056, 3)]
CASES["grouped_mm_dw", "16"] += [(2310, 1900, 1290, 2)]
CASES["grouped_mm_mx4", "16"] += [(1290, 2200, 1058, 2), (2048, 64, 4096, 64)]
CASES["grouped_mm_mx4", "mx4"] += [(1290, 2200, 1088, 2), (2048, 64, 4096, 64)]
CASES["mm_mx4", "16"] += [(2310, 1025, 1058, 1), (11008, 16, 4096, 1)]
CASES["mm_mx4", "mx4"] += [(2310, 1025, 1088, 1), (11008, 16, 4096, 1)]
FLAT = [(op, x, *c) for (op, x), cs in CASES.items() for c in cs]
X_TYPE = {"16": torch.bfloat16, "mx4": torch.uint8}


def kernel(op, x, M, N, K, E):
    """What tells one kernel from another."""
    family, cols, rows, splits = ssg.ssg_mm_select_kernel(op, X_TYPE[x], M, N, K, E)
    return op, x, family, cols, rows, splits > 1


def test_every_kernel_that_is_chosen_has_a_case():
    covered = {kernel(*c) for c in FLAT}
    r = random.Random(7)

    def size(lo, hi):
        return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))

    met = {}
    for _ in range(60000):
        op, x = r.choice(list(CASES))
        M, N, K, E = size(1, 20000), size(1, 8192), size(1, 65536), size(1, 96)
        c = op, x, M, N, max(32, K // 32 * 32) if x == "mx4" else K, 1 if op == "mm_mx4" else E
        met[kernel(*c)] = c
    assert len(met) > 80
    missing = {k: c for k, c in met.items() if k not in covered}
    assert not missing, missing


def test_the_choice_does_not_depend_on_the_16_bit_type():
    for op, x, M, N, K, E in FLAT:
        if x == "16":
            assert (ssg.ssg_mm_select_kernel(op, torch.float16, M, N, K, E) ==
                    ssg.ssg_mm_select_kernel(op, torch.bfloat16, M, N, K, E))


def test_choice_refusals():
    for args, status in (((torch.float32, 8, 8, 8), 4), ((torch.bfloat16, -1, 8, 8), 2)):
        with pytest.raises(ssg.SsgError) as e:
            ssg.ssg_mm_select_kernel("mm_mx4", *args)
        assert e.value.status == status
    for op in ("grouped_mm", "grouped_mm_dx", "grouped_mm_dw"):
        with pytest.raises(ssg.SsgError) as e:
            ssg.ssg_mm_select_kernel(op, torch.uint8, 8, 8, 8)
        assert e.value.status == 4


# ---------------------------------------------------------------- on the device

def sizes_of(E, N, seed):
    """Uneven rows for E experts, some without any; and rows of no expert at both
    ends where there are enough."""
    r = random.Random(seed)
    first, last = (r.randrange(0, 20), r.randrange(0, 20)) if N > 40 * E else (0, 0)
    weight = [0.0 if E > 3 and r.random() < 0.2 else math.exp(r.gauss(0.0, 0.7)) for _ in range(E)]
    weight[r.randrange(E)] += 1.0
    counts = [0] * E
    for e in r.choices(range(E), weight, k=N - first - last):
        counts[e] += 1
    return counts, first


class Mx4:
    """mx4 rows [.., R, K] on the device and their 64-bit values."""

    def __init__(self, gen, shape, K, scales=(118, 124)):
        nb = D.blocks(K)
        code = torch.randint(0, 16, (*shape, nb * 32), generator=gen, device="cuda", dtype=torch.uint8)
        code[..., K:] = 0
        self.code, self.K = code, K
        lo, hi = scales
        self.scales = torch.randint(lo, hi + 1, (*shape, nb), generator=gen, device="cuda", dtype=torch.uint8)

    @property
    def elems(self):
        return self.code[..., 0::2] | (self.code[..., 1::2] << 4)

    def values(self, *at):
        code, s = self.code[at], self.scales[at]
        table = torch.tensor([*D.CODES, *(-D.CODES)], dtype=torch.float64, device="cuda")
        scale = torch.exp2(s.double() - 127.0)
        scale[s == 255] = math.nan
        v = table[code.long()].unflatten(-1, (-1, 32)) * scale[..., None]
        return v.flatten(-2)[..., :self.K]


def product(l, r):
    """l r^T and the sum of magnitudes, in 64 bits."""
    r = r.t().contiguous()
    return (l @ r).cpu().numpy(), (l.abs() @ r.abs()).cpu().numpy()


def randn(gen, shape, dt, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(D.TORCH[dt])


def apart(t):
    """t at odd elements of a larger tensor of NaN."""
    *lead, R, C = t.shape
    big = torch.full((*lead, R + 2, C + 4 - C % 2), math.nan, dtype=t.dtype, device="cuda")
    view = big[..., 1:-1, 1:1 + C]
    view.copy_(t)
    return view


def check_segments(Y, counts, first, length, what, operands, extra=0.0):
    """Rows of each expert against operands(e, rows); the other rows are zero."""
    end = first + sum(counts)
    assert (Y[:first] == 0).all() and (Y[end:] == 0).all(), what
    at = first
    for e, n in enumerate(counts):
        if n:
            ref, mag = product(*operands(e, slice(at, at + n)))
            D.check(Y[at:at + n], ref, mag + extra, length, "%s, expert %d" % (what, e))
        at += n


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("op,x,M,N,K,E", [c for c in FLAT if "mx4" not in c[0]])
def test_16_bit_products(op, x, M, N, K, E, dt):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    X, W, dY = randn(gen, (N, K), dt), randn(gen, (E, M, K), dt, 0.1), randn(gen, (N, M), dt)
    counts, first = sizes_of(E, N, M + K)
    offs = D.offsets(counts, first).cuda()
    few = ssg.ssg_mm_select_kernel(op, D.TORCH[dt], M, N, K, E)[0] == "few"
    for out in ("f32", dt):
        o = dict(out_dtype=D.TORCH[out])
        if op == "grouped_mm":
            for Xv, Wv in [(X, W)] + ([(apart(X), apart(W))] if few else []):
                check_segments(ssg.grouped_mm(Xv, Wv, offs, **o), counts, first, K, "Y %s" % out,
                               lambda e, s: (X[s].double(), W[e].double()))
        elif op == "grouped_mm_dx":
            check_segments(ssg.grouped_mm_dx(dY, W, offs, **o), counts, first, M, "dX %s" % out,
                           lambda e, s: (dY[s].double(), W[e].double().t()))
        else:
            dW, at = ssg.grouped_mm_dw(dY, X, offs, **o), first
            for e, n in enumerate(counts):
                s = slice(at, at + n)
                D.check(dW[e], *product(dY[s].double().t(), X[s].double().t()), n, "dW %s, expert %d" % (out, e))
                at += n


@pytest.mark.gpu
@pytest.mark.parametrize("scales", ["ordinary", "any"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("op,x,M,N,K,E", [c for c in FLAT if "mx4" in c[0] and c[1] == "16"])
def test_mx4_weights(op, x, M, N, K, E, dt, scales):
    """Also with scales that the 16-bit types cannot hold, and rows inside a dword."""
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    X, W = randn(gen, (N, K), dt), Mx4(gen, (E, M), K)
    if scales == "any":
        odd = torch.rand(W.scales.shape, generator=gen, device="cuda") < 0.02
        W.scales[odd] = torch.randint(90, 160, W.scales.shape, generator=gen, device="cuda", dtype=torch.uint8)[odd]
        W.scales[:, M // 2, 0] = 0
    counts, first = (sizes_of(E, N, M + K) if op == "grouped_mm_mx4" else ([N], 0))
    offs = D.offsets(counts, first).cuda()
    few = ssg.ssg_mm_select_kernel(op, D.TORCH[dt], M, N, K, E)[0] == "few"
    for Xv in [X] + ([apart(X)] if few else []):
        for out in ("f32", dt) if scales == "ordinary" else ("f32",):
            o = dict(out_dtype=D.TORCH[out])
            Y = (ssg.mm_mx4(Xv, W.elems[0], W.scales[0], **o) if op == "mm_mx4" else
                 ssg.grouped_mm_mx4(Xv, W.elems, W.scales, offs, **o))
            check_segments(Y, counts, first, K, "Y %s" % out, lambda e, s: (X[s].double(), W.values(e)))


@pytest.mark.gpu
@pytest.mark.parametrize("op,x,M,N,K,E", [c for c in FLAT if c[1] == "mx4"])
def test_mx4_weights_and_activations(op, x, M, N, K, E):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    X, W = Mx4(gen, (N,), K, (120, 130)), Mx4(gen, (E, M), K, (100, 130))
    counts, first = (sizes_of(E, N, M + K) if op == "grouped_mm_mx4" else ([N], 0))
    offs = D.offsets(counts, first).cuda()
    for out in ("f32", "f16", "bf16"):
        o = dict(xscales=X.scales, out_dtype=D.TORCH[out])
        Y = (ssg.mm_mx4(X.elems, W.elems[0], W.scales[0], **o) if op == "mm_mx4" else
             ssg.grouped_mm_mx4(X.elems, W.elems, W.scales, offs, **o))
        check_segments(Y, counts, first, K, "Y %s" % out, lambda e, s: (X.values(s), W.values(e)))


@pytest.mark.gpu
@pytest.mark.parametrize("op,x,M,N,K,E", [c for c in FLAT if "mx4" in c[0]])
def test_a_nan_scale_stays_in_its_row(op, x, M, N, K, E):
    """Of a weight: its column of the expert's rows; of an activation: its row."""
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    W = Mx4(gen, (E, M), K)
    counts, first = (sizes_of(E, N, M + K) if op == "grouped_mm_mx4" else ([N], 0))
    offs = D.offsets(counts, first).cuda()
    e = max(range(E), key=lambda k: counts[k])
    lo = first + sum(counts[:e])
    W.scales[e, M // 3, -1] = 255
    want = torch.zeros(N, M, dtype=torch.bool, device="cuda")
    want[lo:lo + counts[e], M // 3] = True
    kw = {}
    if x == "mx4":
        X = Mx4(gen, (N,), K, (120, 130))
        X.scales[lo, 0] = 255
        X, kw = X.elems, dict(xscales=X.scales)
    else:
        X = randn(gen, (N, K), "bf16")
        X[lo, 0] = math.nan
    want[lo] = True
    Y = (ssg.mm_mx4(X, W.elems[0], W.scales[0], **kw) if op == "mm_mx4" else
         ssg.grouped_mm_mx4(X, W.elems, W.scales, offs, **kw))
    assert torch.equal(torch.isnan(Y), want)
