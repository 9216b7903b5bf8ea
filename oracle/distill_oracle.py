"""fp64 distillation from a teacher's top logits (include/distill.h), from the
definition: whole logits, the list's softmax entry by entry."""

from __future__ import annotations

import numpy as np


def kd_list(t_idx, t_logit, V, T):
    """(valid [N, K], p [N, K], log p [N, K]); p is 0 and log p -inf off the list."""
    t_idx = np.asarray(t_idx, np.int64)
    with np.errstate(over="ignore"):
        t = np.asarray(t_logit, np.float64) / T
    valid = (t_idx >= 0) & (t_idx < V) & (t > -np.inf)
    t = np.where(valid, t, -np.inf)
    m = t.max(1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(t - m)
    z = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        logp = np.where(valid, t - m - np.log(np.where(z > 0, z, 1.0)), -np.inf)
    return valid, np.exp(logp), logp


def kd_forward(X, W, t_idx, t_logit, T):
    """(loss [N], lse [N], y_top [N, K])."""
    y = np.asarray(X, np.float64) @ np.asarray(W, np.float64).T
    V = y.shape[1]
    valid, p, logp = kd_list(t_idx, t_logit, V, T)
    m = (y / T).max(1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(y / T - m).sum(1))
    y_top = np.where(valid, np.take_along_axis(y, np.where(valid, t_idx, 0), 1), 0.0)
    terms = np.where(valid, p * (np.where(valid, logp, 0.0) - (y_top / T - lse[:, None])), 0.0)
    return T * T * terms.sum(1), lse, y_top


def kd_dlogits(X, W, t_idx, t_logit, T, dloss):
    y = np.asarray(X, np.float64) @ np.asarray(W, np.float64).T
    valid, p, _ = kd_list(t_idx, t_logit, y.shape[1], T)
    _, lse, _ = kd_forward(X, W, t_idx, t_logit, T)
    d = np.exp(y / T - lse[:, None])
    rows = np.broadcast_to(np.arange(len(y))[:, None], valid.shape)
    np.add.at(d, (rows[valid], np.asarray(t_idx)[valid]), -p[valid])
    return d * np.where(valid.any(1), T * np.asarray(dloss, np.float64), 0.0)[:, None]


def kd_backward(X, W, t_idx, t_logit, T, dloss):
    d = kd_dlogits(X, W, t_idx, t_logit, T, dloss)
    return d @ np.asarray(W, np.float64), d.T @ np.asarray(X, np.float64)
