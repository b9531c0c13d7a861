"""Every kernel of the 8-bit products, at sizes where the library chooses it, with
ends inside tiles and blocks, against 64-bit definitions."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _fp8 as D
from tests import _mm

F8 = torch.float8_e4m3fn

# (kernel, columns x rows of a workgroup, parts of the contraction), E (0: dense),
# M, K, N, rows of a scale of W, output
CASES = [
    ("few", 16, 16, 1, 0, 300, 1500, 7, 128, "bf16"),
    ("few", 16, 32, 1, 0, 250, 140, 299, 1, "bf16"),
    ("few", 16, 32, 1, 0, 250, 140, 299, 1, "f32"),
    ("few", 32, 16, 1, 0, 8190, 200, 9, 128, "bf16"),
    ("few", 32, 32, 1, 0, 510, 130, 299, 128, "f32"),
    ("few", 64, 32, 1, 0, 1000, 260, 299, 128, "bf16"),
    ("few", 64, 16, 1, 4, 4090, 260, 9, 128, "bf16"),
    ("few", 64, 32, 1, 4, 4090, 140, 45, 128, "f32"),
    ("few", 16, 32, 1, 4, 1000, 200, 45, 1, "bf16"),
    ("tiles", 128, 128, 1, 0, 300, 700, 590, 128, "bf16"),
    ("tiles", 128, 128, 1, 0, 4100, 130, 1020, 128, "f32"),
    ("tiles", 128, 128, 1, 0, 8190, 260, 599, 1, "bf16"),
    ("tiles", 128, 128, 1, 0, 2050, 520, 1020, 1, "f32"),
    ("tiles", 128, 128, 1, 3, 500, 333, 1900, 128, "bf16"),
    ("tiles", 128, 128, 1, 3, 500, 333, 1900, 1, "f32"),
    ("tiles", 128, 128, 4, 0, 250, 2000, 599, 128, "bf16"),
    ("tiles", 128, 128, 4, 0, 250, 1500, 599, 1, "f32"),
    ("tiles", 128, 128, 8, 0, 60, 8100, 599, 1, "bf16"),
    ("tiles", 128, 128, 2, 0, 1000, 3000, 1199, 1, "f32"),
    ("tiles", 128, 128, 8, 2, 120, 4100, 1030, 128, "f32"),
    ("tiles", 128, 128, 1, 0, 1000, 390, 1100, 1, "bf16"),      # four blocks in LDS
    ("tiles", 128, 128, 1, 5, 1000, 390, 2200, 1, "bf16"),
    ("tiles", 256, 256, 1, 0, 4090, 390, 4090, 128, "bf16"),
    ("tiles", 256, 256, 1, 0, 4100, 260, 4300, 128, "bf16"),    # cut in four
    ("tiles", 256, 256, 1, 0, 4100, 260, 5400, 128, "bf16"),     # cut in two
    ("tiles", 256, 256, 1, 4, 2050, 390, 4500, 128, "bf16"),
]


def dtypes(out):
    return D.TORCH[out]


@pytest.mark.parametrize("name,tq,tp,parts,E,M,K,N,wblock,out", CASES)
def test_sizes_take_the_kernel_that_the_next_test_is_of(name, tq, tp, parts, E, M, K, N, wblock, out):
    assert ssg.ssg_mm_fp8_select_kernel(F8, dtypes(out), M, N, K, E, wblock) == (name, tq, tp, parts)


@pytest.mark.gpu
@pytest.mark.parametrize("name,tq,tp,parts,E,M,K,N,wblock,out", CASES)
def test_kernel(name, tq, tp, parts, E, M, K, N, wblock, out):
    g = np.random.default_rng(M + K + N)
    mats = max(E, 1)
    c, s = D.random_fp8(N, K, M + K)
    xv = D.values(c, s.astype(np.float64))
    X, xs = D.elements(c), torch.from_numpy(s).cuda()
    w = [D.random_fp8(M, K, N + K + e, wblock) for e in range(mats)]
    cut = np.sort(g.integers(0, N + 1, mats - 1)) if mats > 1 else np.zeros(0, np.int64)
    offs = np.concatenate([[0], cut, [N]]).astype(np.int32)
    if E:
        offs[-1] = N - 3 if N - 3 >= offs[-2] else offs[-2]     # rows of nobody
    Y = torch.empty(N + 1, M + 3, dtype=dtypes(out), device="cuda").fill_(7.0)
    view = Y[:N, :M]
    if E:
        W = D.elements(np.stack([a for a, _ in w]))
        S = torch.from_numpy(np.stack([b for _, b in w])).cuda()
        ssg.ssg_grouped_mm_fp8(X, W, S, torch.from_numpy(offs).cuda(), view, xscales=xs)
    else:
        ssg.ssg_mm_fp8(X, D.elements(w[0][0]), torch.from_numpy(w[0][1]).cuda(), view, xscales=xs)
    got = Y.cpu()
    assert (got[N] == 7).all() and (got[:, M:] == 7).all()     # nothing beside the output
    for e in range(mats):
        a, b = int(offs[e]), int(offs[e + 1])
        if a == b:
            continue
        wv = D.values(w[e][0], w[e][1].astype(np.float64))
        D.check(got[a:b, :M], xv[a:b] @ wv.T, np.abs(xv[a:b]) @ np.abs(wv).T, K, "%s %s" % (name, e),
                D.coarse(xv[a:b], wv, s[a:b], w[e][1]))
    assert (got[int(offs[-1]):N, :M] == 0).all()
