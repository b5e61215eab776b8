"""The expert router, written from its definition in 64 bits (oracle; test
infrastructure: the library shares no code with it).

Tokens choose the k largest of their E logits (equal logits in the order of
their experts; -inf and NaN never); weights come from the softmax over all
logits; the balance loss is the mean load fraction times the mean probability
per expert, summed.  Masked tokens and tokens without a choice count for
nothing.
"""

from __future__ import annotations

import numpy as np


def _softmax(row):
    """Probabilities of one row with at least one logit above -inf; a NaN or
    +inf makes all of them NaN."""
    m = np.max(np.where(np.isnan(row), -np.inf, row))
    if np.isnan(row).any() or m == np.inf:
        return np.full(row.shape, np.nan)
    e = np.exp(row - m)
    return e / e.sum()


def route(logits, k, mask=None, renorm=True, alpha=0.0):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    index = np.full((T, k), -1, np.int32)
    weight = np.zeros((T, k))
    prob = np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        ranked = sorted((e for e in range(E) if l[t, e] > -np.inf), key=lambda e: (-l[t, e], e))
        if not ranked:
            continue
        n = min(k, len(ranked))
        index[t, :n] = ranked[:n]
        prob[t] = _softmax(l[t])
        w = prob[t, ranked[:n]]
        weight[t, :n] = w / w.sum() if renorm else w
    counts = np.bincount(index[index >= 0], minlength=E).astype(np.int32)
    key = np.where(index < 0, E, index).reshape(-1)
    live = int((index[:, 0] >= 0).sum()) if T else 0
    loss = alpha * E / (k * max(live, 1) ** 2) * float((counts * prob.sum(0)).sum())
    return dict(index=index, weight=weight, counts=counts,
                offsets=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
                order=np.argsort(key, kind="stable").astype(np.int32), live=live,
                prob_sum=prob.sum(0), loss=loss)


def objective(logits, index, counts, live, dweight, dloss, alpha, mask=None, renorm=True):
    """sum(dweight * weight) + dloss * loss, the choice and the counts held
    fixed: the function whose gradient the backward pass returns."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = index.shape[1]
    total = 0.0
    for t in range(T):
        if (mask is not None and not mask[t]) or index[t, 0] < 0:
            continue
        p = _softmax(l[t])
        used = index[t][index[t] >= 0]
        w = p[used] / p[used].sum() if renorm else p[used]
        total += float((dweight[t, :used.size] * w).sum())
        total += dloss * alpha * E / (k * max(live, 1) ** 2) * float((counts * p).sum())
    return total


def gradient(logits, index, counts, live, dweight, dloss, alpha, mask=None, renorm=True):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = index.shape[1]
    d = np.zeros((T, E))
    c = dloss * alpha * E / (k * max(live, 1) ** 2) * np.asarray(counts, np.float64)
    for t in range(T):
        if (mask is not None and not mask[t]) or index[t, 0] < 0:
            continue
        p = _softmax(l[t])
        used = index[t][index[t] >= 0]
        g = dweight[t, :used.size]
        d[t] = p * (c - (p * c).sum())
        if renorm:
            w = p[used] / p[used].sum()
            d[t, used] += w * (g - (w * g).sum())
        else:
            d[t] -= p * (p[used] * g).sum()
            d[t, used] += p[used] * g
    return d
