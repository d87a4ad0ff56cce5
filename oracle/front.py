"""What an MoE layer computes in front of the experts (oracle side, test infrastructure): the residual
RMS norm with its 8-bit output, the router's product and the gate, from their formulas in float64.

* norm:   h = x + r, v = h / sqrt(mean(h^2) + eps) * g; per 32 columns the smallest power of two 2^s with
  max|v| / 2^s <= 448 (``requant_scale_code``) and v / 2^s for the E4M3 codes.
* router: logits = x W^T.
* gate:   s = softmax(l) or 1 / (1 + e^-l); c = s + b, or l itself without a bias; the groups with the
  largest marks (their largest c, or the sum of the two largest c; of s without a bias); the candidates'
  k largest c; their s, over their sum if renormalised, times a scale.  Ties go to the lowest index, -inf
  is never chosen, NaN ranks on top, missing choices are id -1 and weight 0.  Naive loops over rows.
"""
from __future__ import annotations

import numpy as np

from .formats import requant_scale_code


def norm_ref(x, weight, eps, residual=None):
    """float64 (h, v, UE8M0 codes [T, H/32], v over its block's scale) of real arrays [T, H]."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    v = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    T, H = v.shape
    b = v.reshape(T, H // 32, 32)
    code = requant_scale_code(np.abs(b).max(axis=2))
    scaled = b * np.ldexp(1.0, 127 - code.astype(np.int64))[..., None]
    return h, v, code, scaled.reshape(T, H)


def router_ref(x, w):
    return np.asarray(x, np.float64) @ np.asarray(w, np.float64).T


def scores_ref(logits, score):
    l = np.asarray(logits, np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(axis=1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        return e / np.where(np.isneginf(top), 1.0, e.sum(axis=1, keepdims=True))


def _largest(values, n):
    """Indices of the n largest values that are not -inf, NaN on top, the lowest index first among equals."""
    order = sorted((i for i, v in enumerate(values) if not v == -np.inf),
                   key=lambda i: (0, 0.0, i) if np.isnan(values[i]) else (1, -values[i], i))
    return order[:n]


def gate_ref(logits, topk, score="softmax", bias=None, num_groups=1, topk_groups=1, group_score="max",
             renormalize=True, scale=1.0):
    """(int64 [T, k], float64 [T, k])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores_ref(l, score)
    ids = np.full((T, topk), -1, np.int64)
    w = np.zeros((T, topk))
    n = E // num_groups
    for t in range(T):
        c = l[t].copy() if bias is None else s[t] + np.asarray(bias, np.float64)
        c[np.isneginf(l[t])] = -np.inf
        if num_groups > 1:
            marks = np.full(num_groups, -np.inf)
            src = np.where(np.isneginf(c), -np.inf, s[t]) if bias is None and group_score == "top2" else c
            for g in range(num_groups):
                best = _largest(src[g * n:(g + 1) * n], 2 if group_score == "top2" else 1)
                if best:
                    marks[g] = sum(src[g * n + i] for i in best)
            kept = _largest(marks, topk_groups)
            for g in range(num_groups):
                if g not in kept:
                    c[g * n:(g + 1) * n] = -np.inf
        pick = _largest(c, topk)
        ids[t, :len(pick)] = pick
        w[t, :len(pick)] = s[t, pick]
        if renormalize:
            total = w[t].sum()
            w[t] = 0.0 if total == 0 else w[t] / total
        w[t, len(pick):] = 0.0
    return ids, w * scale
