"""The router's choice of experts, its weights and their gradient (FORMAT F27, F28).

TEST INFRASTRUCTURE (see the package docstring). Row by row in FP64 from the definitions; a
choice is made by sorting (key, index) pairs.
"""

import math

import numpy as np


def router_scores(x, score):
    """Scores [E] of one row of logits (FP64): softmax, or the logistic function. -inf scores 0;
    a row of nothing else scores 0 everywhere."""
    x = np.asarray(x, dtype=np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = np.max(x)
    if top == -math.inf:
        return np.zeros_like(x)
    e = np.exp(x - top)
    return e / np.sum(e)


def route_row(x, topk, score="softmax", bias=None, groups=1, group_topk=1, group_top=1,
              renorm=True, scale=1.0):
    """(ids, weights) of one row; ids are -1 where no expert is left."""
    x = np.asarray(x, dtype=np.float64)
    E = len(x)
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    undefined = np.any(np.isnan(x)) or (score == "softmax" and np.any(x == math.inf))
    if not undefined:
        s = router_scores(x, score)
        c = s + b
        undefined = bool(np.any(np.isnan(c[x > -math.inf])))
    if undefined:
        return np.arange(topk), np.full(topk, math.nan)
    open_ = [e for e in range(E) if x[e] > -math.inf and b[e] > -math.inf]
    key = x if bias is None else c  # logits order also where scores round together
    if groups > 1:
        size = E // groups
        part = key if group_top == 1 else c
        totals = []
        for g in range(groups):
            best = sorted((part[e] for e in open_ if e // size == g), reverse=True)[:group_top]
            totals.append((-sum(best), g) if best else (math.inf, g))
        kept = {g for _, g in sorted(totals)[:group_topk]}
        open_ = [e for e in open_ if e // size in kept]
    ids = [e for _, e in sorted((-key[e], e) for e in open_)][:topk]
    if renorm and ids:
        # relative to the largest chosen logit: exact where the scores themselves underflow
        if score == "softmax":
            w = np.exp(x[ids] - np.max(x[ids]))
        else:
            low, top = np.minimum(x[ids], 0.0), min(np.max(x[ids]), 0.0)
            w = np.exp(low - top) / (1.0 + np.exp(-np.abs(x[ids])))
        w = w / np.sum(w)
    else:
        w = s[ids] if ids else np.zeros(0)
    n = topk - len(ids)
    return np.array(ids + [-1] * n), np.concatenate([scale * w, np.zeros(n)])


def expert_route(x, topk, **kw):
    """(ids int64 [T, topk], weights FP64 [T, topk]) of logits [T, E]."""
    rows = [route_row(r, topk, **kw) for r in np.asarray(x, dtype=np.float64)]
    return (np.array([r[0] for r in rows]).reshape(-1, topk),
            np.array([r[1] for r in rows]).reshape(-1, topk))


def expert_route_backward(x, ids, dw, score="softmax", renorm=True, scale=1.0, **_):
    """dlogits [T, E] of the weights of the slots `ids`, the choice held fixed. Weights that are
    renormalised, and sigmoid's, are functions of the slots' logits alone, whatever the others are."""
    x, dw = np.asarray(x, dtype=np.float64), np.asarray(dw, dtype=np.float64)
    out = np.zeros_like(x)
    for t in range(len(x)):
        slots = [k for k in range(len(ids[t])) if ids[t][k] >= 0]
        if not slots:
            continue
        e = [int(ids[t][k]) for k in slots]
        g = scale * dw[t][slots]
        if score == "softmax" and not renorm:
            with np.errstate(invalid="ignore"):
                s = router_scores(x[t], score)
            G = np.zeros(x.shape[1])
            np.add.at(G, e, g)
            out[t] = s * (G - np.sum(s * G))
            continue
        v = x[t][e]
        with np.errstate(invalid="ignore"):
            if score == "softmax":
                r, other = np.exp(v - np.max(v)), 1.0
            else:
                top = min(np.max(v), 0.0) if renorm and np.max(v) > -math.inf else 0.0
                r = np.exp(np.minimum(v, 0.0) - top) / (1.0 + np.exp(-np.abs(v)))
                other = 1.0 / (1.0 + np.exp(np.minimum(v, 700.0)))  # 1 - s
            if renorm:
                r = r / np.sum(r)
                g = g - np.sum(r * g)
            np.add.at(out[t], e, r * g * other)
    return out
