"""64-bit definitions of routing, the order of expert rows, gather and combine,
and the bounds the kernels are held to.  Nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def scores(l, score):
    """float64 [N, E]; zeros for a row of -inf."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(axis=1, keepdims=True, initial=-np.inf)
        e = np.exp(l - np.where(top == -np.inf, 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def rank(v):
    """Sorting keys: larger first, NaN before all."""
    return np.where(np.isnan(v), -np.inf, -np.where(np.isnan(v), 0.0, v)), ~np.isnan(v)


def best(v, live, n):
    """Indices of the n largest live entries of a vector, ties to the lower one."""
    return sorted(live, key=lambda e: ((0, 0.0) if np.isnan(v[e]) else (1, -v[e]), e))[:n]


def route(l, k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0):
    """(weights float64, experts) of float64 logits [N, E]."""
    N, E = l.shape
    S = E // groups
    s = scores(l, score)
    w, out = np.zeros((N, k)), np.full((N, k), -1, dtype=np.int32)
    for n in range(N):
        c = l[n] if bias is None else s[n] + bias
        live = [e for e in range(E) if l[n, e] != -np.inf and (bias is None or bias[e] != -np.inf)]
        if groups > 1:
            of = s[n] if bias is None and group_score == "top2" else c
            total = np.full(groups, -np.inf)
            for g in range(groups):
                top = best(of, [e for e in live if e // S == g], 2 if group_score == "top2" else 1)
                if top:
                    total[g] = sum(of[e] for e in top)
            stay = best(total, range(groups), top_groups)
            live = [e for e in live if e // S in stay]
        pick = best(c, live, k)
        if not pick:
            continue
        out[n, :len(pick)] = pick
        sj = s[n, pick]
        if renorm:
            if score == "sigmoid":
                x = l[n, pick]
                sj = np.exp(-np.logaddexp(0, -x) + np.logaddexp(0, -x).min()) if np.isfinite(x).all() else sj
            else:
                sj = np.exp(l[n, pick] - l[n, pick].max())
            sj = sj / sj.sum()
        w[n, :len(pick)] = sj * scale
    return w, out


def route_grad(dw, l, experts, score="softmax", renorm=True, scale=1.0):
    """(gradient, magnitude of what it is the difference of) of the chosen
    weights with respect to the logits, float64 [N, E]."""
    N, E = l.shape
    s = scores(l, score)
    d, mag = np.zeros((N, E)), np.zeros((N, E))
    for n in range(N):
        js = [j for j, e in enumerate(experts[n]) if 0 <= e < E and l[n, e] != -np.inf]
        if not js:
            continue
        es, g = [int(experts[n, j]) for j in js], dw[n, js] * scale
        x = l[n, es]
        if renorm:
            if score == "sigmoid":
                q = np.exp(-np.logaddexp(0, -x) + np.logaddexp(0, -x).min())
                f = 1.0 / (1.0 + np.exp(x))
            else:
                q, f = np.exp(x - x.max()), 1.0
            q = q / q.sum()
            v, m = q * f * (g - (g * q).sum()), q * f * (np.abs(g) + np.abs(g * q).sum())
        elif score == "sigmoid":
            v = g * s[n, es] / (1.0 + np.exp(x))
            m = np.abs(v)
        else:
            G, A = np.zeros(E), np.zeros(E)
            np.add.at(G, es, g)
            np.add.at(A, es, np.abs(g))
            d[n] = s[n] * (G - (g * s[n, es]).sum())
            mag[n] = s[n] * (A + np.abs(g * s[n, es]).sum())
            continue
        np.add.at(d[n], es, v)
        np.add.at(mag[n], es, m)
    return d, mag


def order(experts, E):
    """(offs, rows, pos) of integer experts [N, k]."""
    flat = experts.reshape(-1)
    offs, rows = [0], []
    for e in range(E):
        rows += np.nonzero(flat == e)[0].tolist()
        offs.append(len(rows))
    pos = np.full(flat.size, -1, dtype=np.int32)
    pos[rows] = np.arange(len(rows))
    rows = rows + [-1] * (flat.size - len(rows))
    return np.array(offs, dtype=np.int32), np.array(rows, dtype=np.int32).reshape(-1), pos.reshape(experts.shape)


def half_step(ref, dtype):
    """Half a step of a type at ref (and of its subnormals)."""
    fi = torch.finfo(dtype)
    return np.abs(ref) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def close(got, ref, tol, what):
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, what
    tol = tol + half_step(np.abs(ref) + tol, got.dtype)
    same = (g == ref) | (np.isnan(g) & np.isnan(ref))
    bad = ~(same | (np.abs(g - ref) <= tol))
    assert not bad.any(), "%s: %d of %d outside, worst %g of the bound" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(g - ref) / np.maximum(tol, 1e-300)))


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TORCH[dtype])
