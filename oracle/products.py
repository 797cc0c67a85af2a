"""Expert products in 8 bits in float64: the tokens' sort by expert and the
weighted way back, quantisation to E4M3 with a power-of-two scale for each group
of 128 values, and the products of such operands.

TEST INFRASTRUCTURE ONLY, like oracle.moe: the product path never uses it.
"""
from __future__ import annotations

import numpy as np

from . import formats as F

BLOCK = 128
_E4M3 = F.e4m3_lut()


def sort_tokens(ids, E):
    """(row_of_slot [T, k], slot_of_row [T * k], seg_start [E + 1]), counted out slot by slot."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    of = [[] for _ in range(E)]
    for s, e in enumerate(flat):
        if 0 <= e < E:
            of[e].append(s)
    row_of_slot = np.full(flat.size, -1, np.int32)
    slot_of_row = np.full(flat.size, -1, np.int32)
    seg_start = np.zeros(E + 1, np.int32)
    r = 0
    for e in range(E):
        for s in of[e]:
            row_of_slot[s], slot_of_row[r] = r, s
            r += 1
        seg_start[e + 1] = r
    return row_of_slot.reshape(ids.shape), slot_of_row, seg_start


def unpermute(y, row_of_slot, w=None):
    """sum_j w[t, j] * y[row], and the same sum of absolute terms."""
    y, rows = np.asarray(y, np.float64), np.asarray(row_of_slot)
    out = np.zeros((rows.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t, j in np.argwhere(rows >= 0):
        term = y[rows[t, j]] * (1.0 if w is None else float(w[t, j]))
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def unpermute_backward(d_out, y, row_of_slot, w):
    """(d_y with NaN in the rows that no slot has, d_w, the sums of d_w's absolute terms)."""
    d_out, y, rows = np.asarray(d_out, np.float64), np.asarray(y, np.float64), np.asarray(row_of_slot)
    d_y = np.full(y.shape, np.nan)
    d_w, mag = np.zeros(rows.shape), np.zeros(rows.shape)
    for t, j in np.argwhere(rows >= 0):
        r = rows[t, j]
        d_y[r] = float(w[t, j]) * d_out[t]
        d_w[t, j] = d_out[t] @ y[r]
        mag[t, j] = np.abs(d_out[t]) @ np.abs(y[r])
    return d_y, d_w, mag


def _group(v):
    """Codes and scale of the values of one group (any shape)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v[~np.isnan(v)])
    e = max(-126, int(F.scale_exponent(a.max() if a.size else 0.0, F.E4M3_MAX)))
    return F.round_to_code(np.ldexp(v, -e), "e4m3"), np.ldexp(1.0, e)


def quantize_rows(x):
    """codes [rows, cols], scales [ceil(cols / 128), rows]."""
    rows, cols = x.shape
    codes, scales = np.empty((rows, cols), np.uint8), np.empty((-(-cols // BLOCK), rows))
    for g in range(scales.shape[0]):
        for r in range(rows):
            codes[r, g * BLOCK:(g + 1) * BLOCK], scales[g, r] = _group(x[r, g * BLOCK:(g + 1) * BLOCK])
    return codes, scales


def quantize_weights(w):
    """codes [E, N, K], scales [E, ceil(N / 128), ceil(K / 128)]."""
    E, N, K = w.shape
    codes, scales = np.empty((E, N, K), np.uint8), np.empty((E, -(-N // BLOCK), -(-K // BLOCK)))
    for e, i, j in np.ndindex(*scales.shape):
        at = (e, slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
        codes[at], scales[e, i, j] = _group(w[at])
    return codes, scales


def padded_rows(rows, E):
    return (rows + 127 * min(rows, E)) // BLOCK * BLOCK


def quantize_cols(x, seg):
    """codes [blocks * 128, cols] and scales [blocks, cols] of the blocks that the segments fill, in order."""
    codes, scales = [], []
    for a, b in zip(seg[:-1], seg[1:]):
        for r in range(a, b, BLOCK):
            part = np.zeros((BLOCK, x.shape[1]))
            n = min(BLOCK, b - r)
            part[:n] = x[r:r + n]
            got = [_group(part[:, c]) for c in range(x.shape[1])]
            codes.append(np.stack([c for c, _ in got], 1))
            scales.append(np.array([s for _, s in got]))
    if not codes:
        return np.empty((0, x.shape[1]), np.uint8), np.empty((0, x.shape[1]))
    return np.concatenate(codes), np.stack(scales)


def values_rows(codes, scales):
    """What row-quantised codes stand for."""
    return _E4M3[codes] * np.repeat(np.asarray(scales, np.float64).T, BLOCK, 1)[:, :codes.shape[1]]


def values_weights(codes, scales):
    _, N, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), BLOCK, 1), BLOCK, 2)[:, :N, :K]
    return _E4M3[codes] * s


def values_cols(codes, scales):
    return _E4M3[codes] * np.repeat(np.asarray(scales, np.float64), BLOCK, 0)


def gemm(x, w, seg, transpose=False):
    """Each expert's rows times its weights (values, not codes), and the sums of
    the absolute terms; NaN in rows outside the segments."""
    w = w if transpose else np.swapaxes(w, 1, 2)
    out, mag = np.full((x.shape[0], w.shape[2]), np.nan), np.full((x.shape[0], w.shape[2]), np.nan)
    for e, (a, b) in enumerate(zip(seg[:-1], seg[1:])):
        out[a:b] = x[a:b] @ w[e]
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e])
    return out, mag


def wgrad(dy, x, seg):
    """dW [E, N, K] from block-aligned values (quantize_cols' order), and the sums of the absolute terms."""
    E = len(seg) - 1
    dw, mag = np.zeros((E, dy.shape[1], x.shape[1])), np.zeros((E, dy.shape[1], x.shape[1]))
    at = 0
    for e, (a, b) in enumerate(zip(seg[:-1], seg[1:])):
        n = -(-(b - a) // BLOCK) * BLOCK
        dw[e] = dy[at:at + n].T @ x[at:at + n]
        mag[e] = np.abs(dy[at:at + n]).T @ np.abs(x[at:at + n])
        at += n
    return dw, mag
