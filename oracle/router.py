"""The router's balance and z losses, their gradients, and the gradients of the weighted combine, in
FP64, written out token by token.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    balance = 1/nseg sum_s E / (k n_s^2) sum_e c_se P_se      z = 1/nseg sum_s 1/n_s sum_t lse_t^2

over the n_s counted tokens of segment s, c_se assignments to expert e, P_se the sum of its
probabilities.  Counts are constants for the gradient.  A token whose logits are all -infinity has
no probabilities and no lse; ids outside [0, E) are not counted.
"""

from __future__ import annotations

import numpy as np


def softmax(logits: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """p [T, E] and lse [T]."""
    l = np.asarray(logits, np.float64)
    mx = l.max(1, keepdims=True)
    none = np.isneginf(mx)
    p = np.exp(l - np.where(none, 0.0, mx))
    s = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(none, 0.0, p / s), np.where(none, 0.0, mx + np.log(s))[:, 0]


def balance(logits, ids, mask=None, offsets=None):
    """dict(loss [2], counts, prob_sums, tokens)."""
    T, E = logits.shape
    k = ids.shape[1]
    off = [0, T] if offsets is None else [int(v) for v in offsets]
    n = len(off) - 1
    p, lse = softmax(logits) if T else (np.zeros((0, E)), np.zeros(0))
    counts, psum, tokens = np.zeros((n, E), np.int64), np.zeros((n, E)), np.zeros(n, np.int64)
    loss = np.zeros(2)
    for s in range(n):
        z = 0.0
        for t in range(off[s], off[s + 1]):
            if mask is not None and not mask[t]:
                continue
            tokens[s] += 1
            psum[s] += p[t]
            z += lse[t] ** 2
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if tokens[s]:
            loss += [E / (k * tokens[s] ** 2) * (counts[s] * psum[s]).sum() / n, z / tokens[s] / n]
    return dict(loss=loss, counts=counts, prob_sums=psum, tokens=tokens)


def balance_backward(logits, ids, counts, tokens, dloss, dtopk_w=None, renorm=False, mask=None, offsets=None):
    """dlogits [T, E]."""
    T, E = logits.shape
    k = ids.shape[1]
    off = [0, T] if offsets is None else [int(v) for v in offsets]
    n = len(off) - 1
    d = np.zeros((T, E))
    p, lse = softmax(logits) if T else (np.zeros((0, E)), np.zeros(0))
    for s in range(n if dloss is not None else 0):
        for t in range(off[s], off[s + 1]):
            if (mask is None or mask[t]) and tokens[s] > 0:
                c = counts[s].astype(np.float64)
                m = float(tokens[s])
                d[t] += dloss[0] * E / (n * k * m * m) * p[t] * (c - (c * p[t]).sum())
                d[t] += dloss[1] * 2 / (n * m) * lse[t] * p[t]
    for t in range(T if dtopk_w is not None else 0):
        if not np.any(dtopk_w[t] != 0):
            continue
        live = [(int(e), float(g)) for e, g in zip(ids[t], dtopk_w[t]) if 0 <= e < E]
        if renorm:
            z = sum(p[t, e] for e, _ in live)
            if z == 0:
                continue
            inner = sum(p[t, e] / z * g for e, g in live)
            for e, g in live:
                d[t, e] += p[t, e] / z * (g - inner)
        else:
            inner = sum(p[t, e] * g for e, g in live)
            d[t] -= p[t] * inner
            for e, g in live:
                d[t, e] += p[t, e] * g
    return d


def combine_backward(dout, Y, token_row, topk_w):
    """(dY [R, H], dtopk_w [T, k]); rows that no token names stay 0."""
    T, k = token_row.shape
    dY, dw = np.zeros(Y.shape), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = token_row[t, j]
            if 0 <= r < len(Y):
                dY[r] = float(topk_w[t, j]) * dout[t].astype(np.float64)
                dw[t, j] = (dout[t].astype(np.float64) * Y[r].astype(np.float64)).sum()
    return dY, dw
