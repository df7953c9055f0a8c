"""What stands around a block's linears, in float64 (oracle side): the norm with
the residual's addition, activations, and routing by scores with a bias and
groups of experts.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Written from the definitions, routing one token at a time.
"""

import numpy as np


def rmsnorm(h, weight, eps):
    """(rstd, y) of h (rows x cols)."""
    h = np.asarray(h, np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
        return rstd, h * rstd[:, None] * np.asarray(weight, np.float64)


def rmsnorm_grad(dy, h, weight, rstd):
    """(dh, dweight) with the given factors."""
    dy, h, f = (np.asarray(t, np.float64) for t in (dy, h, rstd))
    v = h * f[:, None]
    t = dy * np.asarray(weight, np.float64)
    return f[:, None] * (t - v * np.mean(t * v, axis=1, keepdims=True)), np.sum(dy * v, axis=0)


def _sigmoid(u):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-u))


_K, _C = np.sqrt(2.0 / np.pi), 0.044715


def act(z, name):
    z = np.asarray(z, np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * _sigmoid(z)
    return 0.5 * z * (1.0 + np.tanh(_K * (z + _C * z ** 3)))


def act_slope(z, name):
    z = np.asarray(z, np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(z)
        return s + z * s * _sigmoid(-z)
    t = np.tanh(_K * (z + _C * z ** 3))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _K * (1.0 + 3.0 * _C * z * z)


def _scores(row, score):
    """Scores of one token's logits, 0 for a closed expert."""
    if score == "sigmoid":
        return _sigmoid(row)
    if (row == -np.inf).all():
        return np.zeros_like(row)
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.exp(row - np.max(row))
        return z / np.sum(z)


def _order(values, open_):
    """The open indexes by value, largest first: NaN above all, equal ones by index."""
    nan = np.isnan(values)
    return sorted((i for i in range(len(values)) if open_[i]),
                  key=lambda i: (not nan[i], 0.0 if nan[i] else -values[i], i))


def route_groups(logits, topk, bias=None, score="sigmoid", groups=1, topk_groups=None, group_top=2,
                 renorm=True, scale=1.0):
    """(ids, weights): ids -1 and weight 0 where no open expert is left."""
    l = np.asarray(logits, np.float64)
    t, e = l.shape
    keep = groups if topk_groups is None else topk_groups
    ids, w = np.full((t, topk), -1, np.int32), np.zeros((t, topk))
    for i in range(t):
        s = _scores(l[i], score)
        if bias is None and (keep == groups or group_top == 1):
            c = l[i]
        else:
            c = s if bias is None else s + np.asarray(bias, np.float64)
        open_ = (l[i] != -np.inf) & (c != -np.inf)
        if keep < groups:
            size = e // groups
            total, some = np.full(groups, -np.inf), np.zeros(groups, bool)
            for g in range(groups):
                best = [m for m in _order(c, open_) if m // size == g][:group_top]
                some[g] = bool(best)
                if best:
                    total[g] = sum(c[m] for m in best)
            stay = _order(total, some)[:keep]
            open_ = open_ & np.isin(np.arange(e) // size, stay)
        chosen = _order(c, open_)[:topk]
        ids[i, :len(chosen)] = chosen
        w[i, :len(chosen)] = scale * _weights(l[i], s, chosen, score, renorm)
    return ids, w


def _weights(row, s, chosen, score, renorm):
    if not renorm or not chosen:
        return s[chosen]
    with np.errstate(over="ignore", invalid="ignore"):
        # logarithms of the scores (up to a common term): their sum may be below the smallest number
        log = -np.logaddexp(0.0, -row[chosen]) if score == "sigmoid" else row[chosen]
        v = np.exp(log - np.max(log))
        return v / np.sum(v)


def route_groups_grad(logits, ids, dweights, score="sigmoid", renorm=True, scale=1.0):
    """(dlogits, the magnitudes that its differences are of)."""
    l = np.asarray(logits, np.float64)
    d, mag = np.zeros_like(l), np.zeros_like(l)
    for i in range(l.shape[0]):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[i, j] < l.shape[1]]
        if not at:
            continue
        ch = [int(ids[i, j]) for j in at]
        g = scale * np.asarray(dweights[i], np.float64)[at]
        s = _scores(l[i], score)
        w = _weights(l[i], s, ch, score, renorm)
        if score == "sigmoid":
            rest = _sigmoid(-l[i][ch])
            mean, size = (np.sum(w * g), np.sum(w * np.abs(g))) if renorm else (0.0, 0.0)
            d[i, ch] = (g - mean) * w * rest
            mag[i, ch] = (np.abs(g) + size) * w * rest
        elif renorm:
            d[i, ch] = (g - np.sum(w * g)) * w
            mag[i, ch] = (np.abs(g) + np.sum(w * np.abs(g))) * w
        else:
            full = np.zeros_like(s)
            full[ch] = g
            d[i] = s * (full - np.sum(s * full))
            mag[i] = s * (np.abs(full) + np.sum(s * np.abs(full)))
    return d, mag
