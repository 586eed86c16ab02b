"""The routing in 64 bits (numpy on the host), for the operator tests: token by token, by sorting."""

import numpy as np


def _each(f, x):
    """f of every entry, equal entries with equal results (a vector exp may differ from its scalar tail)."""
    u, at = np.unique(x, return_inverse=True)
    with np.errstate(all="ignore"):
        return f(u)[at].reshape(x.shape)


def _sigmoid(u):
    return np.where(u >= 0, 1 / (1 + np.exp(-np.abs(u))), np.exp(-np.abs(u)) / (1 + np.exp(-np.abs(u))))


def scores(l, score):
    if score == "sigmoid":
        return _each(_sigmoid, l)
    m = l.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        p = np.where(np.isneginf(l), 0.0, _each(np.exp, l - np.where(np.isneginf(m), 0.0, m)))
        s = p.sum(axis=1, keepdims=True)
        return np.where(s > 0, p / np.where(s > 0, s, 1), np.where(np.isnan(s), np.nan, 0.0))


def route(l, k, bias=None, groups=1, keep=1, by="max", score="softmax", renorm=True, scale=1.0):
    """(idx, weights, bad): weights in float64, bad the tokens with a NaN."""
    l = l.astype(np.float64)
    n, e = l.shape
    s = scores(l, score)
    dead = np.isneginf(l)
    with np.errstate(all="ignore"):
        choice = np.where(dead, -np.inf, l if bias is None else s + bias.astype(np.float64)[None])
        value = np.where(dead, -np.inf, s) if bias is None and by == "top2" else choice
    bad = np.isnan(choice).any(1) | np.isnan(l).any(1) | ((l == np.inf).any(1) if score == "softmax" else False)
    idx = np.full((n, k), -1, dtype=np.int64)
    w = np.zeros((n, k))
    per = e // groups
    for t in range(n):
        if bad[t]:
            w[t] = np.nan
            continue
        c = choice[t].copy()
        if groups > 1:
            v = -np.sort(-value[t].reshape(groups, per), axis=1)
            g = v[:, 0] + (np.where(np.isneginf(v[:, 1]), 0.0, v[:, 1]) if by == "top2" and per > 1 else 0.0)
            best = np.argsort(-g, kind="stable")[:keep]
            closed = np.ones(groups, dtype=bool)
            closed[best] = False
            c[np.repeat(closed, per)] = -np.inf
        order = np.argsort(-c, kind="stable")[:k]
        order = order[~np.isneginf(c[order])]
        j = len(order)
        idx[t, :j] = order
        if not renorm:
            w[t, :j] = scale * s[t, order]
        elif j:
            x = l[t, order]
            if score == "softmax":
                q = np.exp(x - x.max())
            else:
                b = min(x.max(), 0.0)
                q = np.where(x > 0, 1.0, np.exp(np.minimum(x, 0) - b)) / (1 + np.exp(-np.abs(x)))
            w[t, :j] = scale * q / q.sum()
    return idx, w, bad


def backward(g, l, idx, score, renorm, scale):
    """(grad, size): float64 [n, E] from slots that may repeat; size bounds what its terms sum to before they cancel."""
    l = l.astype(np.float64)
    n, e = l.shape
    s = scores(l, score)
    there = (idx >= 0) & (idx < e)
    at = np.where(there, idx, 0)
    x = np.where(there, np.take_along_axis(l, at, 1), -np.inf)
    with np.errstate(all="ignore"):
        if renorm:
            top = x.max(axis=1, keepdims=True)
            top = np.where(np.isneginf(top), 0.0, top)
            if score == "softmax":
                q = np.exp(x - top)
            else:
                b = np.minimum(top, 0.0)
                q = np.where(x > 0, 1.0, np.exp(np.minimum(x, 0) - b)) / (1 + np.exp(-np.abs(x)))
            d = q.sum(axis=1, keepdims=True)
            share = np.where(d > 0, q / np.where(d > 0, d, 1), 0.0)
        else:
            share = np.where(there, np.take_along_axis(s, at, 1), 0.0)
    gs = np.where(there, scale * g.astype(np.float64), 0.0)
    dot = (gs * share).sum(axis=1, keepdims=True)
    big = (np.abs(gs) * share).sum(axis=1, keepdims=True)
    whole = score == "softmax" and not renorm
    v = share * (gs - (dot if renorm else 0.0))
    size = share * (np.abs(gs) + (big if renorm else 0.0))
    if score == "sigmoid":
        gate = np.where(there, _each(_sigmoid, -np.where(there, x, 0.0)), 0.0)
        v, size = v * gate, size * gate
    grad, bound = np.zeros((n, e)), np.zeros((n, e))
    if whole:
        any_ = there.any(1, keepdims=True)
        grad, bound = np.where(any_, -s * dot, 0.0), np.where(any_, s * big, 0.0)
    for t in range(n):
        for j in range(idx.shape[1]):
            if there[t, j]:
                grad[t, idx[t, j]] += v[t, j]
                bound[t, idx[t, j]] += size[t, j]
    return grad, bound
