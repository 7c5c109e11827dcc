"""Gated projections and their gradients, in binary64 (test oracle).

Test infrastructure: see the package docstring for who may import this.

    g = x Wg^T, u = x Wu^T, h = act(g) u,   W [2I,K], gate rows first
    dgu = (d_h u act'(g), d_h act(g)), d_x = dgu W, d_w = dgu^T x

Each result comes with the largest error that the library's roundings allow:
fp32 sums of n terms in any order, at most 2^-23 of their magnitudes an
addition; the activation within 2^-20; one rounding to the 16-bit type (half a
step, `half`) of h, of dgu, and of the gradients; 24 bits of the factors where
they are saved.
"""
from __future__ import annotations

import math

import numpy as np

HALF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"bfloat16": 2.0 ** -133, "float16": 2.0 ** -25}    # half the smallest step
ADD, EVAL, KEPT = 2.0 ** -23, 2.0 ** -20, 2.0 ** -16
SLOPE = 1.13        # |act'| <= 1.129 and |act''| <= 1 for all three

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(g, name):
    """act(g), act'(g)."""
    if name == "gelu":
        cdf = 0.5 * _erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        with np.errstate(over="ignore"):
            t = np.tanh(c * (g + 0.044715 * g ** 3))
        low = 1.0 / (1.0 + np.exp(np.minimum(-2.0 * c * (g + 0.044715 * g ** 3), 700.0)))
        return g * low, low + g * 0.5 * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    s = 1.0 / (1.0 + np.exp(np.minimum(-g, 700.0)))
    return g * s, s * (1.0 + g * (1.0 - s))


def project(x, w, name):
    """g, u and their error bounds, act(g), act'(g)."""
    i, k = w.shape[0] // 2, x.shape[1]
    gu = x @ w.T
    e = (k + 2) * ADD * (np.abs(x) @ np.abs(w).T)
    a, da = act(gu[:, :i], name)
    return gu[:, :i], gu[:, i:], e[:, :i], e[:, i:], a, da


def forward(x, w, name, dtype):
    """h and its tolerance."""
    _, u, eg, eu, a, _ = project(x, w, name)
    h = a * u
    tol = SLOPE * eg * np.abs(u) + (np.abs(a) + SLOPE * eg) * eu + EVAL * np.abs(h)
    return h, tol + HALF[dtype] * (np.abs(h) + tol) + TINY[dtype]


def factors(x, w, name):
    """(u act'(g), act(g)) and its error before any rounding to 16 bits."""
    g, u, eg, eu, a, da = project(x, w, name)
    f = np.concatenate([u * da, a], 1)
    e = np.concatenate([(np.abs(da) + eg) * eu + np.abs(u) * eg + EVAL * np.abs(u) * SLOPE * (1 + np.abs(g)),
                        SLOPE * eg + EVAL * np.abs(a)], 1)
    return f, e


def backward(d_h, x, w, name, dtype, saved):
    """(d_x, its tolerance, d_w, its tolerance)."""
    half, tiny = HALF[dtype], TINY[dtype]
    f, e = factors(x, w, name)
    if saved:
        e = e + KEPT * (np.abs(f) + e)
    d = np.concatenate([d_h, d_h], 1)
    dgu = d * f
    t = np.abs(d) * e
    t = t + (half + 2 * ADD) * (np.abs(dgu) + t) + tiny
    out = []
    for a, at, b in ((dgu, t, w), (dgu.T, t.T, x)):
        v = a @ b
        tol = at @ np.abs(b) + (a.shape[1] + 2) * ADD * ((np.abs(a) + at) @ np.abs(b))
        out += [v, tol + half * (np.abs(v) + tol) + tiny]
    return tuple(out)
