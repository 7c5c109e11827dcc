"""Routing with its balance loss, rows by group and the weighted return of
the experts' rows, in binary64 from their definitions (test oracle).

Test infrastructure: see the package docstring for who may import this.

* A row is routed if its mask is set and some logit is above -inf.  It
  chooses the k largest logits, ties to the lowest expert, never -inf; slots
  left over hold -1.  Weights: softmax over the chosen logits (renormalize) or
  softmax over all experts at the chosen ones.
* loss = coef * sum_e f_e P_e, f_e = counts_e E / (k n), P_e the mean of the
  softmax over the n routed rows; the counts carry no gradient.
* Rows by group: stable, numbers outside [0, G) last and in no group.
"""
from __future__ import annotations

import numpy as np


def softmax(l: np.ndarray) -> np.ndarray:
    e = np.exp(l - l.max())
    return e / e.sum()


def route(logits, k, mask=None, renormalize=True, coef=0.0):
    """logits fp64 [T,E] -> ids [T,k], weights [T,k], counts [E], n, loss."""
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    counts = np.zeros(E, np.int32)
    prob = np.zeros(E)
    n = 0
    for t in range(T):
        l = logits[t]
        if (mask is not None and not mask[t]) or not np.any(l > -np.inf):
            continue
        n += 1
        chosen = [e for e in sorted(range(E), key=lambda e: (-l[e], e)) if l[e] > -np.inf][:k]
        p = softmax(l)
        w = softmax(l[chosen]) if renormalize else p[chosen]
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w
        counts[chosen] += 1
        prob += p
    loss = 0.0 if n == 0 else coef * float(np.sum(counts * E / (k * n) * (prob / n)))
    return ids, weights, counts, n, loss


def route_value(logits, k, ids, counts, n, renormalize, coef, d_weights, d_loss):
    """The scalar whose gradient route_backward is: the choice, the counts and
    n held fixed."""
    E = logits.shape[1]
    total, prob = 0.0, np.zeros(E)
    for t in range(len(logits)):
        chosen = [int(e) for e in ids[t] if e >= 0]
        if not chosen:
            continue
        p = softmax(logits[t])
        w = softmax(logits[t][chosen]) if renormalize else p[chosen]
        total += float(np.sum(w * d_weights[t, :len(chosen)]))
        prob += p
    return total + (d_loss * coef * float(np.sum(counts * E / (k * n) * (prob / n))) if n else 0.0)


def route_backward(logits, k, ids, counts, n, renormalize, coef, d_weights, d_loss):
    """-> (d_logits [T,E], the sum of the terms' magnitudes [T,E])."""
    T, E = logits.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        chosen = [int(e) for e in ids[t] if e >= 0]
        if not chosen:
            continue
        p = softmax(logits[t])
        dw = d_weights[t, :len(chosen)]
        g = d_loss * coef * counts * E / (k * n) / n
        if renormalize:
            w = softmax(logits[t][chosen])
            d[t, chosen] += w * (dw - np.sum(w * dw))
            mag[t, chosen] += w * (np.abs(dw) + np.sum(w * np.abs(dw)))
        else:
            g = g.copy()
            g[chosen] += dw
        d[t] += p * (g - np.sum(p * g))
        mag[t] += p * (np.abs(g) + np.sum(p * np.abs(g)))
    return d, mag


def group_rows(ids, G):
    key = [int(i) if 0 <= i < G else G for i in ids]
    order = np.array(sorted(range(len(key)), key=key.__getitem__), np.int32)
    positions = np.full(len(key), -1, np.int32)
    offsets = np.zeros(G + 1, np.int32)
    for at, row in enumerate(order):
        if key[row] < G:
            positions[row] = at
            offsets[key[row] + 1:] += 1
    return order, positions, offsets


def combine(y, weights, positions, base=None):
    """-> (out [T,N], the sum of the terms' magnitudes)."""
    T, k = weights.shape
    out = np.zeros((T, y.shape[1])) if base is None else base.astype(np.float64)
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            p = positions[t, j]
            if 0 <= p < len(y):
                out[t] += weights[t, j] * y[p]
                mag[t] += np.abs(weights[t, j] * y[p])
    return out, mag


def combine_weight_gradient(d_out, y, positions):
    """-> (d_weights [T,k], the sum of the terms' magnitudes)."""
    T, k = positions.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = positions[t, j]
            if 0 <= p < len(y):
                dw[t, j] = np.sum(d_out[t] * y[p])
                mag[t, j] = np.sum(np.abs(d_out[t] * y[p]))
    return dw, mag
