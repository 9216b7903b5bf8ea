"""fp64 routing by scores: selection, gates and the gradient of the logits.

Written from the definitions alone (include/route.h): scores are the softmax
or the sigmoid of the logits, experts rank by score plus bias (by logit where
there is none), ties go to the lowest index, a logit of -inf or NaN masks its
expert.  Everything is NumPy fp64, row by row where that reads more plainly.
"""

from __future__ import annotations

import numpy as np


def _clean(logits):
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    return l


def route_log_scores(logits, score: str):
    """log s_e, -inf for masked experts (also where every expert is masked)."""
    l = _clean(logits)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if score == "sigmoid":
            out = np.where(l < 0, l - np.log1p(np.exp(np.minimum(l, 0))), -np.log1p(np.exp(-np.maximum(l, 0))))
        else:
            m = l.max(1, keepdims=True)
            d = np.where(np.isfinite(l), l - np.where(np.isfinite(m), m, 0), -np.inf)
            out = d - np.log(np.exp(d).sum(1, keepdims=True))
    return np.where(np.isfinite(l), out, -np.inf)


def route_select(logits, k, score, bias=None, n_group=1, topk_group=1, group_top=2):
    """topk_idx [N, k]: the experts by rank, the lowest index first on ties."""
    l = _clean(logits)
    N, E = l.shape
    there = np.isfinite(l)
    v = np.exp(route_log_scores(l, score))
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    key = v if bias is not None else l
    idx = np.empty((N, k), np.int64)
    per = E // n_group
    for t in range(N):
        open_ = np.ones(E, bool)
        if n_group > 1:
            strength = np.full(n_group, -np.inf)
            for g in range(n_group):
                best = np.sort(v[t, g * per:(g + 1) * per][there[t, g * per:(g + 1) * per]])[::-1]
                if len(best):
                    strength[g] = best[:group_top].sum()
            keep = sorted(range(n_group), key=lambda g: (-strength[g], g))[:topk_group]
            open_ = np.repeat(np.isin(np.arange(n_group), keep), per)
        order = sorted(np.nonzero(open_)[0], key=lambda e: (not there[t, e], -key[t, e] if there[t, e] else 0.0, e))
        idx[t] = order[:k]
    return idx


def route_gates(logits, idx, score, renorm=True, scale=1.0):
    ls = np.take_along_axis(route_log_scores(logits, score), idx, 1)
    if renorm:
        m = ls.max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0)
        r = np.exp(ls - m)
        z = r.sum(1, keepdims=True)
        return scale * np.where(z > 0, r / np.where(z > 0, z, 1), 0.0)
    return scale * np.exp(ls)


def route_backward(logits, idx, dgates, score, renorm=True, scale=1.0):
    """dL/dlogits [N, E] for dL/dgates, the selection held constant."""
    l = _clean(logits)
    g = route_gates(l, idx, score, renorm, scale)
    dg = np.where(g > 0, np.asarray(dgates, np.float64), 0.0)
    # through log s_e: g = scale s / (renorm ? sum s : 1)
    dls = g * dg
    if renorm:
        dls = dls - g / scale * (g * dg).sum(1, keepdims=True)
    full = np.zeros(l.shape)
    np.add.at(full, (np.arange(len(l))[:, None], idx), dls)
    s = np.exp(route_log_scores(l, score))
    if score == "sigmoid":
        return full * np.where(np.isfinite(l), np.exp(route_log_scores(-np.where(np.isfinite(l), l, 0), "sigmoid")), 0.0)
    # renormalised shares sum to 0 exactly, so the softmax's own sum drops out
    return full if renorm else full - s * full.sum(1, keepdims=True)
