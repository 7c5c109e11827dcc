"""Low-rank adapters of many requests, in binary64 (test oracle).

Test infrastructure: see the package docstring for who may import this.

out[t] = base[t] + scale[g] (x[t] A[g]^T) B[g]^T with g = ids[t]; rows whose
number is outside [0, L) have no adapter.
"""
from __future__ import annotations

import numpy as np


def lora_add(base, x, a, b, ids, scale=None):
    """base [T,N] or None, x [T,K], a [L,r,K], b [L,N,r] -> (out [T,N], the sum
    of the terms' magnitudes [T,N])."""
    T, L, N = len(ids), a.shape[0], b.shape[1]
    out = np.zeros((T, N)) if base is None else base.astype(np.float64)
    mag = np.abs(out)
    for g in range(L):
        rows = np.flatnonzero(np.asarray(ids) == g)
        if len(rows) == 0:
            continue
        s = 1.0 if scale is None else float(scale[g])
        xg, ag, bg = x[rows].astype(np.float64), a[g].astype(np.float64), b[g].astype(np.float64)
        out[rows] += s * (xg @ ag.T) @ bg.T
        mag[rows] += abs(s) * (np.abs(xg) @ np.abs(ag).T) @ np.abs(bg).T
    return out, mag
