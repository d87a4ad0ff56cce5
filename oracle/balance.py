"""Balance of the experts' load and the gate's gradient (oracle side, test infrastructure), from their formulas in
float64, sequence by sequence and row by row."""
from __future__ import annotations

import numpy as np


def spans(T, offsets):
    """[(first row, row behind the last)] of the sequences; None: one of all rows."""
    if offsets is None:
        return [(0, T)]
    o = np.clip(np.asarray(offsets, np.int64), 0, T)
    return [(int(a), int(max(a, b))) for a, b in zip(o, o[1:])]


def row_scores(l, score):
    """(scores, log-sum-exp, whether the row has a candidate) of one row of logits in float64."""
    alive = bool((~np.isneginf(l)).any())
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(np.isneginf(l), 0.0, 1.0 / (1.0 + np.exp(-l))), 0.0, alive
        top = l.max() if alive else 0.0
        e = np.exp(l - top)
        return (e / e.sum() if alive else np.zeros_like(l)), (top + np.log(e.sum()) if alive else 0.0), alive


def row_shares(l, score):
    """Scores over their sum, whatever their size: formed over the largest."""
    s, lse, alive = row_scores(l, score)
    if score == "sigmoid" and alive:
        with np.errstate(all="ignore"):
            top = min(float(np.max(l)), 0.0)
            n = np.where(l >= 0, 1.0, np.exp(np.minimum(l, 0.0) - top)) / (1.0 + np.exp(-np.abs(l)))
            s = n / n.sum()
    return s, lse, alive


def balance_ref(logits, ids, offsets=None, score="softmax"):
    """dict of counts, rows, share, loss, z per sequence."""
    l, ids = np.asarray(logits, np.float64), np.asarray(ids)
    T, E = l.shape
    out = {k: [] for k in ("counts", "rows", "share", "loss", "z")}
    for a, b in spans(T, offsets):
        counts, share, rows, z = np.zeros(E, np.int64), np.zeros(E), 0, 0.0
        for t in range(a, b):
            for e in ids[t]:
                if 0 <= e < E:
                    counts[e] += 1
            p, lse, alive = row_shares(l[t], score)
            rows += alive
            share += p
            z += lse * lse
        share = share / rows if rows else np.zeros(E)
        out["counts"].append(counts)
        out["rows"].append(rows)
        out["share"].append(share)
        out["loss"].append(E * float(counts @ share) / counts.sum() if counts.sum() else 0.0)
        out["z"].append(z / rows if rows else 0.0)
    return {k: np.array(v) for k, v in out.items()}


def objective(logits, ids, counts, rows, d_loss=None, d_z=None, d_topk_w=None, offsets=None, score="softmax", renormalize=True,
              scale=1.0):
    """What gate_grad_ref is the gradient of."""
    l, ids = np.asarray(logits, np.float64), np.asarray(ids)
    T, E = l.shape
    total = 0.0
    for s, (a, b) in enumerate(spans(T, offsets)):
        f = np.asarray(counts[s], np.float64) if d_loss is not None else None
        for t in range(a, b):
            p, lse, alive = row_shares(l[t], score)
            if d_loss is not None and rows[s] and f.sum():
                total += d_loss[s] * E * float(f @ p) / f.sum() / rows[s]
            if d_z is not None and rows[s]:
                total += d_z[s] * lse * lse / rows[s]
            if d_topk_w is not None:
                sc = row_scores(l[t], score)[0]
                w = np.array([sc[e] if 0 <= e < E else 0.0 for e in ids[t]])
                if renormalize and w.sum():
                    w = w / w.sum()
                total += scale * float(w @ np.asarray(d_topk_w[t], np.float64))
    return total


def gate_grad_ref(logits, ids, counts=None, rows=None, d_loss=None, d_z=None, d_topk_w=None, offsets=None, score="softmax",
                  renormalize=True, scale=1.0):
    """float64 [T, E]; NaN in the rows of no sequence, which are not written."""
    l, ids = np.asarray(logits, np.float64), np.asarray(ids)
    T, E = l.shape
    out = np.full((T, E), np.nan)
    for s, (a, b) in enumerate(spans(T, offsets)):
        g = np.zeros(E)
        if d_loss is not None and rows[s] and np.sum(counts[s]):
            g = d_loss[s] * E * np.asarray(counts[s], np.float64) / np.sum(counts[s], dtype=np.float64) / rows[s]
        for t in range(a, b):
            p, lse, alive = row_shares(l[t], score)
            sg = row_scores(l[t], "sigmoid")[0]
            with np.errstate(all="ignore"):
                rest = np.where(l[t] >= 0, np.exp(-np.abs(l[t])), 1.0) / (1.0 + np.exp(-np.abs(l[t])))  # 1 - sigmoid
            r = p * (g - p @ g)
            if score == "sigmoid":
                r = r * rest
            if d_z is not None and rows[s]:
                r = r + p * 2.0 * lse * d_z[s] / rows[s]
            if d_topk_w is not None:
                ok = [(j, int(e)) for j, e in enumerate(ids[t]) if 0 <= e < E and not np.isneginf(l[t, e])]
                if ok:
                    e = np.array([x for _, x in ok])
                    d = scale * np.asarray(d_topk_w[t], np.float64)[[j for j, _ in ok]]
                    if renormalize:
                        top = l[t][e].max() if score == "softmax" else min(l[t][e].max(), 0.0)
                        w = np.exp(l[t][e] - top) if score == "softmax" else \
                            np.where(l[t][e] >= 0, 1.0, np.exp(np.minimum(l[t][e], 0.0) - top)) / (1.0 + np.exp(-np.abs(l[t][e])))
                        w = w / w.sum()
                        d = d - w @ d
                    else:
                        w = p[e] if score == "softmax" else sg[e]
                        if score == "softmax":
                            r = r - p * (w @ d)
                    np.add.at(r, e, w * d * (rest[e] if score == "sigmoid" else 1.0))
            out[t] = np.where(np.isneginf(l[t]), 0.0, r)
    return out
