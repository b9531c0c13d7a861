"""Around the expert-grouped products: which experts a token goes to, the order
of the rows by expert, the copies into that order and the sums out of it, and
the gradients of these.  The names are the package's own:

    weights, experts = ssg.route(logits, k)
    offs, rows, pos = ssg.expert_order(experts, E)
    Xs = ssg.expert_gather(X, pos, rows)           # rows of the grouped products
    Y = ssg.expert_combine(Ys, pos, weights)       # and back

Gradients: route_backward, expert_combine_backward, and for the gather
expert_combine without weights.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _abi
from . import (SsgError, _check, _compiled, _empty, _float, _lib, _mat, _need, _on_device, _raw_stream,
               _same_device, _workspace_size)

__all__ = ["ssg_route", "ssg_route_backward", "ssg_expert_order", "ssg_expert_order_workspace_bytes",
           "ssg_expert_gather", "ssg_expert_combine", "ssg_expert_combine_backward",
           "route", "route_backward", "expert_order", "expert_gather", "expert_combine", "expert_combine_backward"]

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


def _of(t: torch.Tensor, dtype: torch.dtype, name: str) -> torch.Tensor:
    if t.dtype != dtype:
        raise SsgError(_abi.SSG_ERR_DTYPE, "%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _whole(t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> Optional[int]:
    """Address of a contiguous tensor of this type and shape."""
    _of(t, dtype, name)
    _need(tuple(t.shape) == tuple(shape), "%s must be %s" % (name, list(shape)), t)
    if not t.is_contiguous():
        raise SsgError(_abi.SSG_ERR_STRIDE, "%s must be contiguous" % name)
    return _on_device(t, name)


def _named(table, value, name: str) -> int:
    if value not in table:
        raise SsgError(_abi.SSG_ERR_ALGO, "%s must be one of %s, got %r" % (name, ", ".join(table), value))
    return table[value]


# ---------------------------------------------------------------- same-named bindings

def ssg_route(logits, weights, experts, score="softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_score="max", renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    dt, l = _float(logits), _mat(logits, "logits")
    w, e = _mat(_of(weights, torch.float32, "weights"), "weights"), _mat(_of(experts, torch.int32, "experts"), "experts")
    N, E = logits.shape
    k = weights.shape[1]
    _need(weights.shape == (N, k) and experts.shape == (N, k), "shapes of logits, weights, experts", logits, weights,
          experts)
    b = None if bias is None else _whole(bias, torch.float32, (E,), "bias")
    _same_device(logits, weights, experts, bias)
    _check(_lib().ssg_route(dt, N, E, *l, b, _named(_SCORES, score, "score"), k, groups, top_groups,
                            _named(_GROUP_SCORES, group_score, "group_score"), int(renorm), scale, *w, *e,
                            _raw_stream(logits, stream)), "ssg_route")


def ssg_route_backward(dweights, logits, experts, dlogits, score="softmax", renorm: bool = True, scale: float = 1.0,
                       stream=None) -> None:
    dt, l = _float(logits), _mat(logits, "logits")
    w = _mat(_of(dweights, torch.float32, "dweights"), "dweights")
    e, d = _mat(_of(experts, torch.int32, "experts"), "experts"), _mat(_of(dlogits, logits.dtype, "dlogits"), "dlogits")
    N, E = logits.shape
    k = experts.shape[1]
    _need(dweights.shape == (N, k) and experts.shape == (N, k) and dlogits.shape == (N, E),
          "shapes of dweights, logits, experts, dlogits", dweights, logits, experts, dlogits)
    _same_device(logits, dweights, experts, dlogits)
    _check(_lib().ssg_route_backward(dt, N, E, *w, *l, *e, _named(_SCORES, score, "score"), k, int(renorm), scale, *d,
                                     _raw_stream(logits, stream)), "ssg_route_backward")


def ssg_expert_order_workspace_bytes(N: int, k: int, E: int) -> int:
    return int(_lib().ssg_expert_order_workspace_bytes(N, k, E))


def ssg_expert_order(experts, E: int, offs, rows, pos, ws=None, stream=None) -> None:
    e = _mat(_of(experts, torch.int32, "experts"), "experts")
    N, k = experts.shape
    out = (_whole(offs, torch.int32, (E + 1,), "offs"), _whole(rows, torch.int32, (N * k,), "rows"),
           _whole(pos, torch.int32, (N, k), "pos"))
    _same_device(experts, offs, rows, pos)
    s = _raw_stream(experts, stream)
    need = ssg_expert_order_workspace_bytes(N, k, E)
    if ws is not None:
        at, size = _on_device(ws, "ws"), _workspace_size(ws, experts.device)
    else:
        ws = _empty(need, torch.uint8, experts, stream) if need else None
        at, size = (ws.data_ptr() if need else None), need
    _check(_lib().ssg_expert_order(N, k, E, *e, *out, at, size, s), "ssg_expert_order")


def _pairs(pos, rows=None):
    """(N, k, addresses) of an order."""
    _need(pos.dim() == 2, "pos must be 2-D", pos)
    N, k = pos.shape
    at = (_whole(pos, torch.int32, (N, k), "pos"),)
    if rows is not None:
        at += (_whole(rows, torch.int32, (N * k,), "rows"),)
    return N, k, at


def ssg_expert_gather(X, pos, rows, Y, stream=None) -> None:
    dt, x, y = _float(X), _mat(X, "X"), _mat(_of(Y, X.dtype, "Y"), "Y")
    N, k, at = _pairs(pos, rows)
    D = X.shape[1]
    _need(X.shape[0] == N and Y.shape == (N * k, D), "shapes of X, pos, Y", X, pos, Y)
    _same_device(X, pos, rows, Y)
    _check(_lib().ssg_expert_gather(dt, N, k, D, *x, *at, *y, _raw_stream(X, stream)), "ssg_expert_gather")


def ssg_expert_combine(Y, pos, O, weights=None, stream=None) -> None:
    dt, y, out, o = _float(Y), _mat(Y, "Y"), _float(O), _mat(O, "O")
    N, k, at = _pairs(pos)
    D = Y.shape[1]
    _need(Y.shape[0] == N * k and O.shape == (N, D), "shapes of Y, pos, O", Y, pos, O)
    w = (None, 0)
    if weights is not None:
        w = _mat(_of(weights, torch.float32, "weights"), "weights")
        _need(weights.shape == (N, k), "shapes of weights, pos", weights, pos)
    _same_device(Y, pos, O, weights)
    _check(_lib().ssg_expert_combine(dt, out, N, k, D, *y, *at, *w, *o, _raw_stream(Y, stream)), "ssg_expert_combine")


def ssg_expert_combine_backward(dO, Y, pos, rows, weights, dY, dweights, stream=None) -> None:
    dt, o, y = _float(dO), _mat(dO, "dO"), _mat(_of(Y, dO.dtype, "Y"), "Y")
    N, k, at = _pairs(pos, rows)
    D = dO.shape[1]
    w, dw = (_mat(_of(t, torch.float32, n), n) for t, n in ((weights, "weights"), (dweights, "dweights")))
    d = _mat(_of(dY, dO.dtype, "dY"), "dY")
    _need(dO.shape[0] == N and Y.shape == (N * k, D) and dY.shape == Y.shape and weights.shape == (N, k) and
          dweights.shape == (N, k), "shapes of dO, Y, pos, weights, dY, dweights", dO, Y, pos, weights, dY, dweights)
    _same_device(dO, Y, pos, rows, weights, dY, dweights)
    _check(_lib().ssg_expert_combine_backward(dt, N, k, D, *o, *y, *at, *w, *d, *dw, _raw_stream(dO, stream)),
           "ssg_expert_combine_backward")


# ---------------------------------------------------------------- calls that allocate their outputs

def route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
          group_score: str = "max", renorm: bool = True, scale: float = 1.0,
          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(weights fp32 [N, k], experts int32 [N, k]) of logits [N, E] (fp16, bf16 or
    fp32): the k experts with the largest score ("softmax" or "sigmoid" of the
    logits, plus bias [E] fp32 if given) in descending order, ties to the lower
    number, out of the top_groups best of `groups` groups of neighbouring
    experts (by their largest score or, "top2", the sum of their two largest).
    A weight is scale times the expert's score without the bias, with renorm
    divided by the sum over the chosen ones.  A logit (or bias) of -inf: never
    chosen; slots left over get expert -1 and weight 0."""
    if stream is None:
        done = _compiled().route(logits, k, score, bias, groups, top_groups, group_score, renorm, scale)
        if done is not None:
            return done
    _need(logits.dim() == 2, "logits must be 2-D", logits)
    _need(0 <= k <= logits.shape[1], "k = %d of the experts" % k, logits)
    weights = _empty((logits.shape[0], k), torch.float32, logits, stream)
    experts = _empty((logits.shape[0], k), torch.int32, logits, stream)
    ssg_route(logits, weights, experts, score, bias, groups, top_groups, group_score, renorm, scale, stream)
    return weights, experts


def route_backward(dweights, logits, experts, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
                   stream=None) -> torch.Tensor:
    """Gradient of route's weights with respect to the logits, in their type."""
    if stream is None:
        done = _compiled().route_backward(dweights, logits, experts, score, renorm, scale)
        if done is not None:
            return done
    _need(logits.dim() == 2 and experts.dim() == 2, "logits and experts must be 2-D", logits, experts)
    dlogits = _empty(logits.shape, logits.dtype, logits, stream)
    ssg_route_backward(dweights, logits, experts, dlogits, score, renorm, scale, stream)
    return dlogits


def expert_order(experts, E: int, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(offs [E + 1], rows [N * k], pos [N, k]) of experts [N, k], all int32: the
    pairs n * k + j sorted by expert, in their own order within one.  Rows
    offs[e] .. offs[e + 1] - 1 are expert e's, rows[r] is the pair of row r, pos
    the row of a pair; -1 for pairs whose expert is not 0 .. E - 1, and for as
    many rows at the end."""
    if stream is None:
        done = _compiled().expert_order(experts, E)
        if done is not None:
            return done
    _need(experts.dim() == 2, "experts must be 2-D", experts)
    N, k = experts.shape
    _need(0 <= E < 1 << 20, "E = %d" % E, experts)
    offs = _empty((E + 1,), torch.int32, experts, stream)
    rows, pos = _empty((N * k,), torch.int32, experts, stream), _empty((N, k), torch.int32, experts, stream)
    ssg_expert_order(experts, E, offs, rows, pos, stream=stream)
    return offs, rows, pos


def expert_gather(X, pos, rows, stream=None) -> torch.Tensor:
    """[N * k, D]: row pos[n, j] is X[n]; rows of nobody are zeros."""
    if stream is None:
        done = _compiled().expert_gather(X, pos, rows)
        if done is not None:
            return done
    _need(X.dim() == 2 and pos.dim() == 2, "X and pos must be 2-D", X, pos)
    Y = _empty((pos.numel(), X.shape[1]), X.dtype, X, stream)
    ssg_expert_gather(X, pos, rows, Y, stream)
    return Y


def expert_combine(Y, pos, weights=None, out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """[N, D]: the sum over j of weights[n, j] (None: 1) times Y[pos[n, j]], in Y's
    type or fp32; fp32 sums."""
    if stream is None:
        done = _compiled().expert_combine(Y, pos, weights, out_dtype)
        if done is not None:
            return done
    _need(Y.dim() == 2 and pos.dim() == 2, "Y and pos must be 2-D", Y, pos)
    O = _empty((pos.shape[0], Y.shape[1]), out_dtype or Y.dtype, Y, stream)
    ssg_expert_combine(Y, pos, O, weights, stream)
    return O


def expert_combine_backward(dO, Y, pos, rows, weights, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dY, dweights) of expert_combine(Y, pos, weights) from dO [N, D]: row
    pos[n, j] of dY is weights[n, j] dO[n] (rows of nobody are zeros), dweights[n, j]
    the product of dO[n] and Y[pos[n, j]]."""
    if stream is None:
        done = _compiled().expert_combine_backward(dO, Y, pos, rows, weights)
        if done is not None:
            return done
    _need(Y.dim() == 2 and weights.dim() == 2, "Y and weights must be 2-D", Y, weights)
    dY, dw = _empty(Y.shape, Y.dtype, Y, stream), _empty(weights.shape, torch.float32, Y, stream)
    ssg_expert_combine_backward(dO, Y, pos, rows, weights, dY, dw, stream)
    return dY, dw
