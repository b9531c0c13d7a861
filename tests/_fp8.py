"""64-bit definitions of the 8-bit format with a scale for each block of 128 and of
its products.  Nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def blocks(n):
    return -(-n // 128)


# the magnitudes of the codes 0 .. 126, ascending
CODES = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8)])[:127]


def nearest(q):
    """Code (sign in bit 7) of the e4m3 number nearest to float64 q, ties to the even
    code; NaN is 127."""
    mag = np.abs(np.where(np.isnan(q), 0.0, q))
    hi = np.searchsorted(CODES, mag).clip(1, 126)
    lo = hi - 1
    below, above = mag - CODES[lo], CODES[hi] - mag
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (np.where(np.isnan(q), 127, code) | (np.signbit(q).astype(np.int64) << 7)).astype(np.uint8)


def quantize(a, block=1):
    """(codes, scales float64) of float64 [R, K]."""
    R, K = a.shape
    codes = np.zeros((R, K), dtype=np.uint8)
    scales = np.zeros((R if block == 1 else blocks(R), blocks(K)))
    for i in range(scales.shape[0]):
        r = slice(i * block, (i + 1) * block)
        for b in range(scales.shape[1]):
            c = slice(b * 128, (b + 1) * 128)
            part = a[r, c]
            top = np.abs(np.where(np.isnan(part), 0.0, part)).max()
            s = float(np.maximum(np.float32(top) / np.float32(448), np.float32(2.0 ** -126)))
            scales[i, b] = s
            with np.errstate(invalid="ignore"):
                codes[r, c] = nearest(part / s)
    return codes, scales


def values(codes, scales):
    """float64 values."""
    v = np.where((codes & 127) == 127, np.nan, CODES[np.minimum(codes & 127, 126)]) * np.where(codes >> 7, -1.0, 1.0)
    R, K = codes.shape
    s = scales if scales.shape[0] == R else np.repeat(scales, 128, axis=0)[:R]
    return v * np.repeat(s, 128, axis=1)[:, :K]


def codes_of(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def coarse(xv, wv, xs, ws):
    """What the 8-bit matrix instruction may lose, for values [N, K], [M, K] and their
    scales.  It adds eight neighbouring products aligned to the largest sum of their
    exponents, E, and cuts each at 2^(E - 13): a product that is not the largest is
    off by less than 2^(E - 13), seven of eight, and 2^E is at most the product of
    the largest magnitudes of the eight (a subnormal counts as 2^-6, its exponent).
    So 7 * 2^-13 of the sum of these products bounds the loss.  (K is padded with
    zeros to whole eights.)"""
    def tops(v, s):
        s = s if s.shape[0] == v.shape[0] else np.repeat(s, 128, axis=0)[:v.shape[0]]
        s = np.repeat(s, 128, axis=1)[:, :v.shape[1]]
        m = np.where(v == 0, 0.0, np.maximum(np.abs(v), 2.0 ** -6 * s))
        m = np.pad(m, ((0, 0), (0, -m.shape[1] % 8)))
        return m.reshape(m.shape[0], m.shape[1] // 8, 8).max(axis=2)
    return 7 * 2.0 ** -13 * (tops(xv, xs.astype(np.float64)) @ tops(wv, ws.astype(np.float64)).T)


def check(got, ref, mag, K, what, loss=0.0):
    """Products of e4m3 numbers are exact in fp32 (8 bits of fraction); a block's sum
    is off by at most 128 steps of 2^-23 of its magnitudes (a whole step an addition,
    so truncating adders count), the two scales' product by half a step, each
    multiply-add of a block by one step of the magnitudes so far, and joining the
    partial sums by 16: K + blocks + 16 steps.  The output adds half a step, and a
    16-bit one what the 8-bit instruction may lose."""
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, what
    tol = (K + blocks(K) + 16) * 2.0 ** -23 * mag
    if got.dtype != torch.float32:
        fi = torch.finfo(got.dtype)
        tol = tol + loss
        tol = tol + (np.abs(ref) + tol) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    else:
        tol = tol + 2.0 ** -149
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %g of the bound" % (
        what, bad.sum(), bad.size, (np.abs(g - ref) / np.maximum(tol, 1e-300)).max())


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TORCH[dtype])


def random_fp8(rows, K, seed, block=1, lo=0, hi=127):
    """Random codes (no NaN) of magnitudes lo .. hi - 1 and scales of magnitudes 2^-4 .. 2^4."""
    g = np.random.default_rng(seed)
    codes = g.integers(lo, hi, size=(rows, K)).astype(np.uint8) | (g.integers(0, 2, size=(rows, K)) << 7).astype(np.uint8)
    n = rows if block == 1 else blocks(rows)
    return codes, np.exp2(g.uniform(-4, 4, size=(n, blocks(K)))).astype(np.float32)


def elements(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(torch.float8_e4m3fn)
