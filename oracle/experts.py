"""Oracle of the experts' routing (numpy, float64), one token after the other."""

import numpy as np


def _ranked(values):
    """Indices of what can be picked (above -infinity), best first: NaN above all numbers, ties by the lower index."""
    v = np.asarray(values, np.float64)
    nan = np.isnan(v)
    by = np.lexsort((np.arange(len(v)), np.where(nan, 0.0, -v), ~nan))
    return by[v[by] != -np.inf].tolist()


def scores(l, kind):
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        if (l == -np.inf).all():
            return np.zeros_like(l)
        e = np.where(l == -np.inf, 0.0, np.exp(l - (np.nan if np.isnan(l).any() else l.max())))
        return e / e.sum()


def route_token(l, top, kind="softmax", bias=None, groups=1, keep=None, pairs=False, renormalize=True, scale=1.0):
    """One token's float64 logits -> (ids, weights), both `top` long."""
    E, keep = len(l), groups if keep is None else keep
    s = scores(l, kind)
    by_logit = bias is None and not (pairs and groups > 1)
    with np.errstate(invalid="ignore"):
        c = l.copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    c[l == -np.inf] = -np.inf
    if groups > 1:
        size = E // groups
        value = []
        for g in range(groups):
            part = c[g * size : (g + 1) * size]
            best = [part[i] for i in _ranked(part)[: 2 if pairs else 1]]
            value.append(sum(best) if best else -np.inf)
        kept = _ranked(value)[:keep]
        for g in range(groups):
            if g not in kept:
                c[g * size : (g + 1) * size] = -np.inf
    picked = _ranked(c)[:top]
    ids, w = np.full(top, -1, np.int32), np.zeros(top)
    ids[: len(picked)] = picked
    of = s[picked]
    if renormalize:
        total = of.sum()
        of = of * 0.0 if total == 0 else of / total
    w[: len(picked)] = of * scale
    return ids, w


def order(ids, E):
    """ids [M, top] -> (offsets, rows of the sorted choices, places)."""
    M, top = ids.shape
    of = [[] for _ in range(E)]
    for m in range(M):
        for j in range(top):
            if ids[m, j] >= 0:
                of[ids[m, j]].append((m, j))
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in of])]).astype(np.int32)
    places, rows = np.full((M, top), -1, np.int32), []
    for m, j in [x for part in of for x in part]:
        places[m, j] = len(rows)
        rows.append(m)
    return offsets, np.asarray(rows, np.int32), places


def route(logits, top, valid=None, **kw):
    """float64 logits [M, E] -> (ids, weights float64, offsets, rows, places)."""
    ids, w = np.full((len(logits), top), -1, np.int32), np.zeros((len(logits), top))
    for m, l in enumerate(logits):
        if valid is None or valid[m]:
            ids[m], w[m] = route_token(l, top, **kw)
    return (ids, w, *order(ids, logits.shape[1]))


def combine(y, places, weights, base=None):
    """(sum, sum of magnitudes) in float64."""
    M, top = places.shape
    out, size = np.zeros((M, y.shape[1])), np.zeros((M, y.shape[1]))
    for m in range(M):
        for j in range(top):
            if 0 <= places[m, j] < len(y):
                term = float(weights[m, j]) * y[places[m, j]]
                out[m] += term
                size[m] += np.abs(term)
    if base is not None:
        out, size = out + base, size + np.abs(base)
    return out, size
