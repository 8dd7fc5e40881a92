"""Routing by scores in fp64 (numpy, one token at a time): the definition that the GPU kernels are
checked against (LightLLM PR #1687, call-order paragraph: grouped top-k and renormalisation inside
`experts()`; the score, bias and group rule are arguments).

  score   sigmoid(l), or the softmax over the experts that are in
  order   score + bias, or the logits without a bias; ties to the lower expert
  weight  scale * score / (sum of the chosen scores), or scale * score
  out     a logit of NaN or -inf: no part at all; a bias of NaN or -inf: not chosen (+inf counts
          as the largest f32)
"""
from __future__ import annotations

import numpy as np

BIG = float(np.finfo(np.float32).max)


def scores(l, kind):
    """(scores, who is in) of one token's logits."""
    l = np.asarray(l, dtype=np.float64)
    there = l > -np.inf  # false for NaN
    l = np.where(there, np.minimum(l, BIG), -BIG)  # (out: a value that overflows nothing)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))),
                         np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    else:
        s = np.exp(l - l[there].max()) * there if there.any() else np.zeros_like(l)
        s = s / s.sum() if there.any() else s
    return np.where(there, s, 0.0), there


def route_token(l, k, kind, bias=None, n_group=1, topk_group=1, group_score="max", renorm=True,
                scale=1.0):
    """(ids, weights in fp64, in) of one token."""
    E = len(l)
    s, there = scores(l, kind)
    there = there & bias_in(bias, E)  # the bias moves the choice alone: the softmax has them all
    if bias is None:
        choice, order = s, np.minimum(np.asarray(l, dtype=np.float64), BIG)
    else:
        b = np.minimum(np.where(bias_in(bias, E), bias, 0.0).astype(np.float64), BIG)
        choice = order = s + b
    allowed = np.ones(E, dtype=bool)
    if topk_group < n_group:
        size = E // n_group
        value = []
        for g in range(n_group):
            ids = [e for e in range(g * size, (g + 1) * size) if there[e]]
            by = order if group_score == "max" else choice
            v = sorted((by[e] for e in ids), reverse=True)
            if not v:
                value.append(-np.inf)
            elif group_score == "max" or len(v) == 1:
                value.append(v[0])
            else:
                value.append(v[0] + v[1])
        taken = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
        allowed = np.isin(np.arange(E) // size, taken)
    first = sorted((e for e in range(E) if allowed[e] and there[e]), key=lambda e: (-order[e], e))
    ids = (first + [e for e in range(E) if allowed[e] and not there[e]])[:k]
    live = there[ids]
    w = np.where(live, s[ids], 0.0)
    if renorm:
        w = w / w.sum() if w.sum() > 0 else w
    return np.array(ids, dtype=np.int32), scale * w, live


def bias_in(bias, E):
    return np.ones(E, dtype=bool) if bias is None else np.asarray(bias) > -np.inf


def route(logits, k, kind, capacity=0, **how):
    """(ids [T, k], weights [T, k] rounded to f32, keep [T, k]) with the capacity: an expert keeps
    the `capacity` largest weights, ties to the earlier token."""
    got = [route_token(l, k, kind, **how) for l in np.asarray(logits, dtype=np.float64)]
    ids = np.stack([g[0] for g in got])
    w = np.stack([g[1] for g in got]).astype(np.float32)
    keep = np.stack([g[2] for g in got]).astype(np.uint8)
    if capacity > 0:
        for e in np.unique(ids):
            t, j = np.nonzero((ids == e) & (keep > 0))
            drop = np.lexsort((t, -w[t, j]))[capacity:]
            keep[t[drop], j[drop]] = 0
    return ids, w, keep


def backward(logits, ids, w, dw, kind, renorm=True, scale=1.0):
    """dlogits [T, E] in fp64, and the sum of the absolute terms of each value."""
    logits = np.asarray(logits, dtype=np.float64)
    out, size = np.zeros_like(logits), np.zeros_like(logits)
    for t, l in enumerate(logits):
        s, there = scores(l, kind)
        at, g = np.asarray(ids[t]), np.asarray(dw[t], dtype=np.float64)
        live = np.asarray(w[t]) != 0  # an expert that was out, or a weight that vanished
        at, g = at[live], g[live]
        v = s[at]
        if renorm and len(at):
            ds = scale * (g / v.sum() - (g * v).sum() / v.sum() ** 2)
            da = scale * (np.abs(g) / v.sum() + (np.abs(g) * v).sum() / v.sum() ** 2)
        else:
            ds, da = scale * g, scale * np.abs(g)
        if kind == "sigmoid":
            x = np.minimum(l[at], BIG)
            with np.errstate(over="ignore"):
                slope = v / (1 + np.exp(x))
            out[t, at], size[t, at] = ds * slope, da * slope
        else:
            d, a = np.zeros_like(l), np.zeros_like(l)
            d[at], a[at] = ds, da
            finite = l < np.inf  # (+inf counts as a number that it does not move)
            out[t] = s * (d - (d * s).sum()) * finite
            size[t] = s * (a + (a * s).sum()) * finite
    return out, size
