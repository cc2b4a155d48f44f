"""Plain 64-bit form of the routing by scores, row by row, for the tests."""
import math

import numpy as np


def _better(a, ia, b, ib):
    """Whether value a at index ia comes before b at ib: NaN last, the lower index on ties."""
    if math.isnan(a) or math.isnan(b):
        return ia < ib if math.isnan(a) and math.isnan(b) else math.isnan(b)
    return a > b or (a == b and ia < ib)


def _rank(values):
    """Indices of `values` from the first choice to the last."""
    nan = np.isnan(values)
    key = np.where(nan, 0.0, -values)
    return np.lexsort((np.arange(len(values)), key, nan))


def scores_of(row, sigmoid):
    l = row.astype(np.float64)
    s = np.zeros(l.size)
    live = ~np.isneginf(l)
    with np.errstate(all="ignore"):
        if sigmoid:
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
        elif live.any():
            e = np.exp(l[live] - np.fmax.reduce(l[live]))
            s[live] = e / e.sum()
    return s


def route(logits, k, sigmoid, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0,
          bias=None):
    """(ids, weights in 64 bits, counts, offsets, perm_tok, inv_row) of logits [T][E]."""
    T, E = logits.shape
    gs = E // groups
    ids = np.empty((T, k), np.int32)
    w = np.empty((T, k))
    for t in range(T):
        s = scores_of(logits[t], sigmoid)
        c = s if bias is None else s + bias.astype(np.float64)
        c = np.where(np.isneginf(logits[t]), -np.inf, c)
        inside = np.arange(E)
        if topk_groups < groups:
            gv = np.empty(groups)
            for g in range(groups):
                own = c[g * gs:(g + 1) * gs]
                gv[g] = sum(own[i] for i in _rank(own)[:group_top])
            kept = sorted(_rank(gv)[:topk_groups])
            inside = np.concatenate([np.arange(g * gs, (g + 1) * gs) for g in kept])
        ids[t] = inside[_rank(c[inside])[:k]]
        v = s[ids[t]]
        if renorm:
            d = v.sum()
            v = np.zeros(k) if d == 0 else v / d
        w[t] = v * np.float64(np.float32(scale))
    flat = ids.reshape(-1)
    rows = np.argsort(flat, kind="stable")
    inv = np.empty(T * k, np.int32)
    inv[rows] = np.arange(T * k)
    counts = np.bincount(flat, minlength=E).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return ids, w, counts, offsets, (rows // k).astype(np.int32), inv.reshape(T, k)
