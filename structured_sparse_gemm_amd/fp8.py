"""8-bit floats (e4m3) with an fp32 scale for each block of 128, and their products:

    w, ws = ssg.fp8_quantize(W, block=128)         # weights: 128 x 128
    Y = ssg.mm_fp8(X, w, ws)                       # X fp16 / bf16, rounded in the call
    x, xs = ssg.fp8_quantize(X)                    # or beforehand, 1 x 128
    Y = ssg.mm_fp8(x, w, ws, xscales=xs)

The gradients of a linear layer are products of the same kind, of operands
quantised along the other direction:

    wt, wts = ssg.fp8_quantize(W, block=128, transpose=True)
    dX = ssg.mm_fp8(dY, wt, wts)
    dyt, dyts = ssg.fp8_quantize(dY, transpose=True)
    xt, xts = ssg.fp8_quantize(X, transpose=True)
    dW = ssg.mm_fp8(dyt, xt, xts, xscales=dyts)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _abi
from . import (_FLOAT, SsgError, _check, _compiled, _empty, _float, _lib, _mat, _need, _offsets, _on_device, _out,
               _raw_stream, _same_device, _stack, _workspace_size)

__all__ = ["ssg_fp8_scale_cols", "ssg_fp8_quantize", "ssg_fp8_dequantize", "ssg_mm_fp8", "ssg_mm_fp8_workspace_bytes",
           "ssg_grouped_mm_fp8", "ssg_grouped_mm_fp8_workspace_bytes", "ssg_mm_fp8_select_kernel",
           "fp8_quantize", "fp8_dequantize", "mm_fp8", "grouped_mm_fp8"]

FP8 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return (n + 127) // 128


def ssg_fp8_scale_cols(K: int) -> int:
    return int(_lib().ssg_fp8_scale_cols(K))


def _elements(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != FP8:
        raise SsgError(_abi.SSG_ERR_DTYPE, "%s must be %s, got %s" % (name, FP8, t.dtype))
    return t


def _scales(t: torch.Tensor, rows: int, cols: int, name: str, mats: Optional[int] = None):
    """(rows to a scale, (address, strides of rows, blocks and matrices)) of the
    scales of rows x cols elements: one for each row, or for each 128."""
    if t.dtype != torch.float32:
        raise SsgError(_abi.SSG_ERR_DTYPE, "%s must be fp32, got %s" % (name, t.dtype))
    lead = () if mats is None else (mats,)
    shape, nb = tuple(t.shape), _blocks(cols)
    if shape == (*lead, rows, nb):
        block = 1
    else:
        block = 128
        _need(shape == (*lead, _blocks(rows), nb), "%s must be %s or %s" % (
            name, [*lead, rows, nb], [*lead, _blocks(rows), nb]), t)
    # the stride of a single row or block means nothing
    *mat, row, blk = (1 if n == 1 else s for n, s in zip(t.shape, t.stride()))
    return block, (_on_device(t, name), row, blk, *mat)


def _as_stack(t: torch.Tensor, name: str):
    """(address, row stride, stride) of a matrix or a stack."""
    if t.dim() == 2:
        return (*_mat(t, name), 0)
    return _stack(t, name)


def _fp8_operands(A, elems, scales, transpose: bool):
    _elements(elems, "elems")
    _need(A.dim() in (2, 3), "the matrix must be 2-D or 3-D", A)
    a, e = _as_stack(A, "the matrix"), _as_stack(elems, "elems")
    *lead, R, K = A.shape
    er, ec = (K, R) if transpose else (R, K)
    _need(tuple(elems.shape) == (*lead, er, ec), "shapes of the matrix, elems", A, elems)
    block, s = _scales(scales, er, ec, "scales", lead[0] if lead else None)
    _same_device(A, elems, scales)
    return (lead[0] if lead else 1, R, K), a, e, block, (s if lead else (*s, 0))


# ---------------------------------------------------------------- same-named bindings

def ssg_fp8_quantize(A, elems, scales, transpose: bool = False, stream=None) -> None:
    dt = _float(A)
    sizes, a, e, block, s = _fp8_operands(A, elems, scales, transpose)
    _check(_lib().ssg_fp8_quantize(dt, *sizes, *a, block, int(transpose), *e, *s, _raw_stream(A, stream)),
           "ssg_fp8_quantize")


def ssg_fp8_dequantize(elems, scales, D, stream=None) -> None:
    dt = _float(D)
    sizes, d, e, block, s = _fp8_operands(D, elems, scales, False)
    _check(_lib().ssg_fp8_dequantize(dt, *sizes, *e, block, *s, *d, _raw_stream(D, stream)), "ssg_fp8_dequantize")


def _x_operands(X, xscales):
    """(type, (address, row stride), (address, strides) of the scales)."""
    _need(X.dim() == 2, "X must be 2-D", X)
    if xscales is None:
        if X.dtype == FP8:
            raise SsgError(_abi.SSG_ERR_FORMAT, "X of %s needs xscales" % (FP8,))
        return _float(X), _mat(X, "X"), (None, 0, 0)
    _elements(X, "X")
    block, s = _scales(xscales, *X.shape, "xscales")
    _need(block == 1, "xscales must have a row for each of X", X, xscales)
    return _abi.SSG_E4M3, _mat(X, "X"), s


def _mm_fp8_operands(X, W, wscales, xscales):
    _elements(W, "W")
    _need(X.dim() == 2 and W.dim() == 2 and X.shape[1] == W.shape[1], "shapes of X, W", X, W)
    x, xa, xs = _x_operands(X, xscales)
    M, K = W.shape
    block, ws = _scales(wscales, M, K, "wscales")
    _same_device(X, W, wscales, xscales)
    return (x, M, X.shape[0], K, *xa, *xs, *_mat(W, "W"), block, *ws)


def _grouped_mm_fp8_operands(X, W, wscales, offs, xscales):
    _elements(W, "W")
    _need(X.dim() == 2 and W.dim() == 3 and X.shape[1] == W.shape[2], "shapes of X, W", X, W)
    x, xa, xs = _x_operands(X, xscales)
    E, M, K = W.shape
    block, ws = _scales(wscales, M, K, "wscales", E)
    _same_device(X, W, wscales, offs, xscales)
    return (x, E, M, X.shape[0], K, *xa, *xs, *_stack(W, "W"), block, *ws, _offsets(offs, E))


def ssg_mm_fp8_workspace_bytes(X, W, wscales, xscales=None, out_dtype: torch.dtype = torch.float32) -> int:
    x, *ops = _mm_fp8_operands(X, W, wscales, xscales)
    return int(_lib().ssg_mm_fp8_workspace_bytes(x, _FLOAT.get(out_dtype, -1), *ops))


def ssg_grouped_mm_fp8_workspace_bytes(X, W, wscales, offs, xscales=None, out_dtype: torch.dtype = torch.float32) -> int:
    x, *ops = _grouped_mm_fp8_operands(X, W, wscales, offs, xscales)
    return int(_lib().ssg_grouped_mm_fp8_workspace_bytes(x, _FLOAT.get(out_dtype, -1), *ops))


def _run(name: str, operands, Y, out, ws, stream) -> None:
    """_run_with_workspace, whose workspace here depends on the output's type too."""
    fn, s = getattr(_lib(), name), _raw_stream(Y, stream)
    x, y, ops = operands[0], _float(Y), operands[1:]
    if ws is not None:
        size = _workspace_size(ws, Y.device)
        _check(fn(x, y, *ops, *out, _on_device(ws, "ws"), size, s), name)
        return
    rc = fn(x, y, *ops, *out, None, _abi.SSG_WS_ASK, s)
    if rc == _abi.SSG_ERR_WORKSPACE:
        need = int(getattr(_lib(), name + "_workspace_bytes")(x, y, *ops))
        ws = _empty(need, torch.uint8, Y, stream)
        rc = fn(x, y, *ops, *out, ws.data_ptr(), need, s)
    if rc:
        _check(rc, name)


def ssg_mm_fp8(X, W, wscales, Y, xscales=None, ws=None, stream=None) -> None:
    ops = _mm_fp8_operands(X, W, wscales, xscales)
    _run("ssg_mm_fp8", ops, Y, _out(Y, "Y", X.shape[0], W.shape[0], X), ws, stream)


def ssg_grouped_mm_fp8(X, W, wscales, offs, Y, xscales=None, ws=None, stream=None) -> None:
    ops = _grouped_mm_fp8_operands(X, W, wscales, offs, xscales)
    _run("ssg_grouped_mm_fp8", ops, Y, _out(Y, "Y", X.shape[0], W.shape[1], X), ws, stream)


def ssg_mm_fp8_select_kernel(x: torch.dtype, out_dtype: torch.dtype, M: int, N: int, K: int, E: int = 0,
                             block: int = 128) -> Tuple[str, int, int, int]:
    """("few" or "tiles", columns and rows of the output a workgroup owns, parts of
    the contraction) of the kernel that mm_fp8 (E = 0) or grouped_mm_fp8 takes."""
    k = (ctypes.c_int64 * 4)()
    dt = _abi.SSG_E4M3 if x == FP8 else _FLOAT.get(x, -1)
    _check(_lib().ssg_mm_fp8_select_kernel(dt, _FLOAT.get(out_dtype, -1), block, E, M, N, K, k), "ssg_mm_fp8_select_kernel")
    return ("tiles" if k[0] else "few",) + tuple(k[1:])


# ---------------------------------------------------------------- calls that allocate their outputs

def fp8_quantize(A, block: int = 1, transpose: bool = False, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(elements, scales) of A [R, K] or a stack [E, R, K]: float8_e4m3fn of the same
    shape and fp32 scales, for each row and 128 columns ([.., R, ceil(K / 128)]) or,
    block=128, each 128 rows and 128 columns ([.., ceil(R / 128), ceil(K / 128)]).
    transpose: those of A's transpose.  A scale is max(amax / 448, 2^-126), an
    element the nearest to A / scale.  Rows of the elements begin at 16 bytes, and
    the scales of rows are stored by blocks, as the products read them."""
    if block not in (1, 128):
        raise SsgError(_abi.SSG_ERR_FORMAT, "%r rows to a scale (1 or 128)" % (block,))
    if stream is None:
        done = _compiled().fp8_quantize(A, block, transpose)
        if done is not None:
            return done
    _need(A.dim() in (2, 3), "A must be 2-D or 3-D", A)
    *lead, R, K = A.shape
    if transpose:
        R, K = K, R
    elems = _empty((*lead, R, (K + 15) // 16 * 16), FP8, A, stream)[..., :K]
    if block == 1:
        scales = _empty((*lead, _blocks(K), (R + 3) // 4 * 4), torch.float32, A, stream)[..., :R].transpose(-1, -2)
    else:
        scales = _empty((*lead, _blocks(R), _blocks(K)), torch.float32, A, stream)
    ssg_fp8_quantize(A, elems, scales, transpose, stream)
    return elems, scales


def fp8_dequantize(elems, scales, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values of e4m3 elements [R, K] or [E, R, K] with their scales, in `dtype`."""
    if stream is None:
        done = _compiled().fp8_dequantize(elems, scales, dtype)
        if done is not None:
            return done
    D = _empty(elems.shape, dtype, elems, stream)
    ssg_fp8_dequantize(elems, scales, D, stream)
    return D


def mm_fp8(X, W, wscales, xscales=None, out_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """X W^T with W [M, K] of float8_e4m3fn and its scales (for each 128 x 128 or
    each row and 128): X [N, K] the same with xscales [N, ceil(K / 128)], or fp16,
    bf16, fp32, then rounded as by fp8_quantize.  Returns [N, M] in out_dtype; the sums
    are fp32's for every output type and number of rows."""
    if stream is None:
        done = _compiled().fp8_product(X, xscales, W, wscales, None, out_dtype)
        if done is not None:
            return done
    _need(X.dim() == 2 and W.dim() == 2, "X and W must be 2-D", X, W)
    Y = _empty((X.shape[0], W.shape[0]), out_dtype, X, stream)
    ssg_mm_fp8(X, W, wscales, Y, xscales=xscales, stream=stream)
    return Y


def grouped_mm_fp8(X, W, wscales, offs, xscales=None, out_dtype: torch.dtype = torch.float32,
                   stream=None) -> torch.Tensor:
    """Rows offs[e] .. offs[e + 1] - 1 of X times W[e]^T, W [E, M, K] (see mm_fp8);
    rows of no expert are zero."""
    if stream is None:
        done = _compiled().fp8_product(X, xscales, W, wscales, offs, out_dtype)
        if done is not None:
            return done
    _need(X.dim() == 2 and W.dim() == 3, "X must be 2-D, W 3-D", X, W)
    Y = _empty((X.shape[0], W.shape[1]), out_dtype, X, stream)
    ssg_grouped_mm_fp8(X, W, wscales, offs, Y, xscales=xscales, stream=stream)
    return Y
