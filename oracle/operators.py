"""The operators around the routed experts in float64: the residual's addition
with the root-mean-square norm and its gradient, routing with score functions
and groups and the gradient of its weights, and the combine's gradient with
respect to those weights.

TEST INFRASTRUCTURE ONLY, like oracle.moe: the product path never uses it.
"""
from __future__ import annotations

import numpy as np

from .moe import sigmoid_fp32


def rmsnorm(x, residual, weight, eps):
    """(h, y) = (x + r, h * (mean(h^2) + eps)^-1/2 * w), unrounded."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return h, y


def rmsnorm_backward(dy, h, weight, dh_in, eps):
    """Gradient of sum(dy * y) with respect to h (plus dh_in) and to the weight."""
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, weight))
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    g = dy * w
    dh = r * g - h * r ** 3 * (g * h).mean(axis=1, keepdims=True)
    return dh + (0.0 if dh_in is None else np.asarray(dh_in, np.float64)), (dy * h * r).sum(axis=0)


def scores(logits, softmax):
    """Scores of the experts that can be chosen, float64; 0 where the logit is
    -inf or NaN and where the score is below e^-700."""
    l = np.asarray(logits, np.float64)
    dead = np.isnan(l) | np.isneginf(l)
    if not softmax:
        with np.errstate(over="ignore", invalid="ignore"):
            return np.where(dead | (l < -700), 0.0, 1.0 / (1.0 + np.exp(-l)))
    l = np.where(dead, -np.inf, l)
    top = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(dead | (l < top - 700), 0.0, np.where(l == top, 1.0, np.exp(l - top)))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def route_grouped(logits, bias, k, softmax=False, n_group=1, topk_group=1, renormalize=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k]); empty slots are -1 and 0."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    s = scores(logits, softmax)
    if bias is None:
        key = logits.copy()
    else:
        s32 = s.astype(np.float32) if softmax else sigmoid_fp32(logits)
        key = s32 + np.asarray(bias, np.float32)[None, :]
    key = np.where(np.isnan(logits) | np.isneginf(logits) | np.isnan(key), np.float32(-np.inf), key)
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    per = E // n_group
    for t in range(T):
        row = key[t].copy()
        if n_group > 1:
            of_group = []
            for g in range(n_group):
                best = np.sort(row[g * per:(g + 1) * per])[::-1]
                two = bias is not None and per > 1 and best[1] > -np.inf
                of_group.append(best[0] + best[1] if two else best[0])
            keep = np.argsort(-np.array(of_group, np.float32), kind="stable")[:topk_group]
            for g in range(n_group):
                if g not in keep:
                    row[g * per:(g + 1) * per] = -np.inf
        order = np.argsort(-row, kind="stable")[:k]
        order = order[row[order] > -np.inf]
        n = len(order)
        ids[t, :n] = order
        w[t, :n] = s[t, order]
        total = w[t].sum()
        if renormalize and total > 0:
            w[t] /= total
    return ids, w * scale


def route_weights(logits, ids, softmax=False, renormalize=True, scale=1.0):
    """The weights of given ids as a function of float64 logits."""
    s = scores(logits, softmax)
    ok = (ids >= 0) & (ids < s.shape[1])
    w = np.where(ok, np.take_along_axis(s, np.where(ok, ids, 0), axis=1), 0.0)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return w * scale


def route_backward(d_w, logits, ids, softmax=False, renormalize=True, scale=1.0):
    """d_logits [T, E]: the chain rule through route_weights, row by row."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, softmax)
    out = np.zeros((T, E))
    for t in range(T):
        d_s = np.zeros(E)  # gradient with respect to each expert's score
        ok = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        total = sum(s[t, ids[t, j]] for j in ok)
        dot = sum(float(d_w[t, j]) * scale * s[t, ids[t, j]] for j in ok)
        for j in ok:
            g = float(d_w[t, j]) * scale
            if not renormalize:
                d_s[ids[t, j]] += g
            elif total > 0:
                d_s[ids[t, j]] += (g - dot / total) / total
        # the softmax's common term sum(d_s * s) is 0 for renormalised weights, which do not
        # change with it: left out there, its rounding would stand at every unchosen expert
        common = (d_s * s[t]).sum() if softmax and not renormalize else 0.0
        out[t] = s[t] * (d_s - common) if softmax else d_s * s[t] * (1.0 - s[t])
    return out


def combine_backward(d_out, y, ids, E, rsf=1.0):
    """d_w [T, k]; the y rows of masked slots are not looked at."""
    T, k = ids.shape
    out = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                out[t, j] = rsf * np.dot(np.asarray(y[t * k + j], np.float64), np.asarray(d_out[t], np.float64))
    return out
