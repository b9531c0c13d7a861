"""64-bit definitions for the mx4 format and the expert-grouped products, and
the error bounds the kernels are held to.  Nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def blocks(K: int) -> int:
    return (K + 31) // 32


def mx4_quantize(a: np.ndarray):
    """(elements, scales) of float64 rows [R, K], element by element from the
    definition: nearest of the eight magnitudes, ties to the even code."""
    R, K = a.shape
    nb = blocks(K)
    v = np.zeros((R, nb * 32))
    v[:, :K] = a
    v = v.reshape(R, nb, 32)
    nan = np.isnan(v).any(axis=2)
    top = np.abs(np.where(np.isnan(v), 0.0, v)).max(axis=2)
    e = np.full(top.shape, -127, dtype=np.int64)
    fin = np.isfinite(top) & (top > 0)
    e[fin] = np.maximum(np.frexp(top[fin])[1] - 1 - 2, -127)
    e[np.isinf(top)] = 126                              # the exponent field of an infinity, 255, less 2 and 127
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.abs(np.where(np.isnan(v), 0.0, v)) / np.exp2(e.astype(np.float64))[:, :, None]
    q = np.minimum(q, 6.0)
    best = np.zeros(q.shape, dtype=np.int64)
    dist = np.abs(q - CODES[0])
    for c in range(1, 8):
        d = np.abs(q - CODES[c])
        take = (d < dist) | ((d == dist) & (c % 2 == 0))
        best = np.where(take, c, best)
        dist = np.where(take, d, dist)
    code = best | (np.signbit(v).astype(np.int64) << 3)
    code[nan] = 0
    code = code.reshape(R, nb * 32)
    scales = np.where(nan, 255, e + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scales


def mx4_values(elems: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """Float64 values of the last two dimensions (elements, scales)."""
    code = np.stack([elems & 15, elems >> 4], axis=-1).reshape(*elems.shape[:-1], -1)
    v = CODES[code & 7] * np.where(code >> 3, -1.0, 1.0)
    s = np.exp2(scales.astype(np.float64) - 127.0)
    s = np.where(scales == 255, np.nan, s)
    return (v * np.repeat(s, 32, axis=-1))[..., :K]


def segments(offs, N):
    """(expert, first row, end row) of every expert."""
    return [(e, int(offs[e]), int(offs[e + 1])) for e in range(len(offs) - 1)]


def grouped(X, W, offs):
    """(Y, sum of magnitudes) in float64: rows of an expert times its W^T, zeros elsewhere."""
    Y = np.zeros((X.shape[0], W.shape[1]))
    S = np.zeros_like(Y)
    for e, a, b in segments(offs, X.shape[0]):
        Y[a:b] = X[a:b] @ W[e].T
        S[a:b] = np.abs(X[a:b]) @ np.abs(W[e]).T
    return Y, S


def grouped_dx(dY, W, offs):
    return grouped(dY, np.swapaxes(W, 1, 2), offs)


def grouped_dw(dY, X, offs):
    E = len(offs) - 1
    D = np.zeros((E, dY.shape[1], X.shape[1]))
    S = np.zeros_like(D)
    for e, a, b in segments(offs, X.shape[0]):
        D[e] = dY[a:b].T @ X[a:b]
        S[e] = np.abs(dY[a:b]).T @ np.abs(X[a:b])
    return D, S


def check(got: torch.Tensor, ref: np.ndarray, mag: np.ndarray, length: int, what: str):
    """Products of 16-bit (or mx4) values are exact in fp32; a sum of `length` of
    them in any order is off by at most length steps of 2^-23 of the sum of
    magnitudes (a whole step an addition, so truncating adders count), plus
    16 for joining partial sums.  A 16-bit output adds half a step of its own
    (and of its subnormals)."""
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, what
    tol = (length + 16) * 2.0 ** -23 * mag
    if got.dtype != torch.float32:
        fi = torch.finfo(got.dtype)
        tol = tol + (np.abs(ref) + tol) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    else:
        tol = tol + 2.0 ** -149
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %g of the bound" % (
        what, bad.sum(), bad.size, (np.abs(g - ref) / np.maximum(tol, 1e-300)).max())


def offsets(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32)


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TORCH[dtype])


def random_mx4(shape, seed, lo=118, hi=124):
    """Random codes and scale bytes in lo .. hi of [.., R, K]."""
    *lead, K = shape
    g = np.random.default_rng(seed)
    nb = blocks(K)
    code = g.integers(0, 16, size=(*lead, nb * 32))
    code[..., K:] = 0
    e = (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)
    return e, g.integers(lo, hi + 1, size=(*lead, nb)).astype(np.uint8)
