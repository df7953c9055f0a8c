"""Routing, token exchange and gradient clipping in float64 (oracle side).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Written from the definitions, one token at a time: the topk largest logits
(ties to the lowest expert, -inf never chosen), softmax weights over the
chosen or all logits, the stable order of the slots by expert, the weighted
sum back and the derivatives of each.
"""

import numpy as np


def route(logits, topk, renorm):
    """(ids, weights): ids -1 and weight 0 where no open expert is left."""
    l = np.asarray(logits, np.float64)
    t, e = l.shape
    ids = np.full((t, topk), -1, np.int32)
    w = np.zeros((t, topk))
    for i in range(t):
        nan = np.isnan(l[i])
        rank = np.where(nan, np.inf, l[i])
        # NaN above everything, then by value, then by index
        order = sorted(range(e), key=lambda x: (not nan[x], -rank[x], x))
        order = [x for x in order if not l[i, x] == -np.inf][:topk]
        if not order:
            continue
        ids[i, :len(order)] = order
        w[i, :len(order)] = softmax(l[i], order if renorm else None)[order]
    return ids, w


def softmax(row, chosen=None):
    """exp(row) over its sum; with chosen, over the sum of those, zero elsewhere."""
    with np.errstate(invalid="ignore"):
        z = np.exp(row - np.max(row))
    if chosen is not None:
        z = np.where(np.isin(np.arange(len(row)), chosen), z, 0.0)
    return z / z.sum()


def route_grad(logits, ids, dweights, renorm):
    l = np.asarray(logits, np.float64)
    d = np.zeros_like(l)
    for i in range(l.shape[0]):
        sel = [j for j in range(ids.shape[1]) if ids[i, j] >= 0]
        if not sel:
            continue
        ch = [int(ids[i, j]) for j in sel]
        p = softmax(l[i], ch if renorm else None)
        # w_j = p[ch_j]; the Jacobian of a softmax is diag(p) - p p^T
        for j, e in zip(sel, ch):
            d[i] += float(dweights[i, j]) * p[e] * ((np.arange(l.shape[1]) == e) - p)
    return d


def sort(ids, experts):
    """(offsets, pos, src) of the stable order by expert, dropped slots last."""
    flat = [int(v) for v in np.asarray(ids).reshape(-1)]
    src = [s for e in range(experts) for s, v in enumerate(flat) if v == e]
    offsets = [0]
    for e in range(experts):
        offsets.append(offsets[-1] + sum(v == e for v in flat))
    src += [s for s, v in enumerate(flat) if not 0 <= v < experts]
    pos = np.zeros(len(flat), np.int32)
    for r, s in enumerate(src):
        pos[s] = r if r < offsets[-1] else ~r
    return (np.array(offsets, np.int64), pos.reshape(np.asarray(ids).shape),
            np.array(src, np.int32))


def dispatch(x, pos):
    t, k = pos.shape
    rows = np.zeros((t * k, x.shape[1]))
    for i in range(t):
        for j in range(k):
            if pos[i, j] >= 0:
                rows[pos[i, j]] = x[i]
    return rows


def combine(rows, pos, weights=None):
    """(y, sum of the magnitudes of y's terms)."""
    t, k = pos.shape
    y, mag = np.zeros((t, rows.shape[1])), np.zeros((t, rows.shape[1]))
    for i in range(t):
        for j in range(k):
            if pos[i, j] >= 0:
                term = rows[pos[i, j]] * (1.0 if weights is None else float(weights[i, j]))
                y[i] += term
                mag[i] += np.abs(term)
    return y, mag


def combine_grad(dy, rows, pos, weights):
    """(drows, dweights, sum of the magnitudes of dweights' terms)."""
    t, k = pos.shape
    drows, dw, mag = np.zeros(rows.shape), np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            if pos[i, j] >= 0:
                drows[pos[i, j]] = float(weights[i, j]) * dy[i]
                dw[i, j] = np.dot(dy[i], rows[pos[i, j]])
                mag[i, j] = np.dot(np.abs(dy[i]), np.abs(rows[pos[i, j]]))
    return drows, dw, mag


def grad_clip(grads, max_norm, eps):
    """(norm, clipped) in float64."""
    norm = np.sqrt(sum(np.sum(np.asarray(g, np.float64) ** 2) for g in grads))
    coef = max_norm / (norm + eps)
    coef = coef if not coef > 1.0 else 1.0
    with np.errstate(invalid="ignore"):
        return norm, [np.asarray(g, np.float64) * coef for g in grads]
