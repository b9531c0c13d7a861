"""Sums of the 8-bit products: fp32's for every kernel and every output type, also
where large terms cancel, so that a row's result does not depend on how many others
are multiplied with it.  The outputs are held to the bound of fp32 sums and half a
step of their own type, nothing else."""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from tests import _fp8 as D
from tests import _mm

F8 = torch.float8_e4m3fn
pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# M, K, N, rows to a scale of W, kernel: one for each kernel of many rows, whole tiles
# and ends inside tiles and blocks
SHAPES = [(500, 1000, 590, 128, ("tiles", 128)), (500, 1000, 590, 1, ("tiles", 128)), (4100, 390, 4090, 128, ("tiles", 256)),
          (4090, 390, 4500, 128, ("tiles", 256)), (4100, 390, 5400, 128, ("tiles", 256)), (300, 1000, 40, 128, ("few", None))]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K,N,wblock,kernel", SHAPES)
def test_sums_of_any_magnitudes(M, K, N, wblock, kernel, out):
    """Codes of every magnitude: products of 2^-18 to 2^17 next to each other."""
    if out != "f32":
        chosen = ssg.ssg_mm_fp8_select_kernel(F8, D.TORCH[out], M, N, K, 0, wblock)
        assert chosen[0] == kernel[0] and kernel[1] in (None, chosen[1])
    cx, sx = D.random_fp8(N, K, 1)
    cw, sw = D.random_fp8(M, K, 2, wblock)
    sx, sw = np.full_like(sx, 2.0 ** -6), np.full_like(sw, 2.0 ** -6)      # (fp16 holds the sums)
    xv, wv = D.values(cx, sx.astype(np.float64)), D.values(cw, sw.astype(np.float64))
    Y = ssg.mm_fp8(D.elements(cx), D.elements(cw), dev(sw), xscales=dev(sx), out_dtype=D.TORCH[out])
    D.check(Y, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, K, "mm_fp8 -> " + out)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("wblock", [1, 128])
@pytest.mark.parametrize("M,N", [(300, 700), (4100, 4090)])
def test_small_terms_beside_large_ones_that_cancel(M, N, wblock, out):
    """One pair of products in each block of 128 is 256 * 256 and -256 * 256, the others are
    2^-6 to 2^1: whatever the order of a sum, its parts are below 2^17 and multiples of
    2^-6, which fp32 holds, so the sums are exact, and the outputs their rounding."""
    K = 256
    g = np.random.default_rng(3)
    x, w = np.exp2(g.integers(-3, 1, size=(N, K))), np.exp2(g.integers(-3, 2, size=(M, K)))
    x[:, 0::128], x[:, 1::128], w[:, :2], w[:, 128:130] = 256.0, -256.0, 256.0, 256.0
    ref = x @ w.T
    ones = torch.ones(N, 2).cuda(), torch.ones(M if wblock == 1 else D.blocks(M), 2).cuda()
    Y = ssg.mm_fp8(dev(x).to(F8), dev(w).to(F8), ones[1], xscales=ones[0], out_dtype=D.TORCH[out])
    want = torch.from_numpy(ref).to(D.TORCH[out])
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_grouped_sums_of_any_magnitudes(out):
    M, K, sizes = 520, 390, [900, 0, 1300, 700]
    N, offs = sum(sizes), _mm.offsets(sizes)
    cx, sx = D.random_fp8(N, K, 1)
    parts = [D.random_fp8(M, K, 5 + e, 128) for e in range(len(sizes))]
    sx = np.full_like(sx, 2.0 ** -6)
    sw = np.stack([np.full_like(s, 2.0 ** -6) for _, s in parts])
    xv = D.values(cx, sx.astype(np.float64))
    wv = np.stack([D.values(c, s.astype(np.float64)) for (c, _), s in zip(parts, sw)])
    ref, mag = _mm.grouped(xv, wv, offs.tolist())
    Y = ssg.grouped_mm_fp8(D.elements(cx), D.elements(np.stack([c for c, _ in parts])), dev(sw), offs.cuda(),
                           xscales=dev(sx), out_dtype=D.TORCH[out])
    D.check(Y, ref, mag, K, "grouped_mm_fp8 -> " + out)
