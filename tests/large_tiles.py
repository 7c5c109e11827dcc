"""Sizes whose products run on 256 x 256 tiles, and the oracle's formulas on the
device for outputs of that size (binary64 torch, element by element)."""
import math

import torch

from oracle import gated as og
from oracle import w4 as ow

# (M, I, K), and what its products' plans are: forward, d_x, d_w.  "L": large tiles, "Ln":
# in n ranges of K, "L+": large tiles for the columns of whole rounds, the others by a
# plan of their own; "": any other shape.
GATED = [((1003, 4099, 1536), ("L", "", "L")), ((3773, 547, 3815), ("L3", "L", "L3")),
         ((732, 2869, 3761), ("L3", "L5", "L")), ((4000, 2203, 2056), ("L+", "L", "L")),
         ((1170, 3780, 2310), ("L", "L5", "L+")), ((4428, 549, 4337), ("L2", "L+", "L3"))]
# (M, N, K) of 4-bit products; groups of 32, 64 and 128
W4 = [((1837, 7338, 384), "L"), ((702, 3730, 3200), "L5"), ((572, 7546, 2816), "L2"),
      ((4369, 3860, 1152), "L+")]


def act(g, name):
    """act(g), act'(g)."""
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if name == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g)
    s, t = torch.sigmoid(z), torch.sigmoid(-z)
    return g * s, s * (1.0 + g * t * dz)


def rounded(v, tol, dtype):
    return tol + og.HALF[dtype] * (v.abs() + tol) + og.TINY[dtype]


def project(x, w):
    """g, u and their error bounds."""
    i, k = w.shape[0] // 2, x.shape[1]
    gu, e = x @ w.t(), (k + 2) * og.ADD * (x.abs() @ w.abs().t())
    return gu[:, :i], gu[:, i:], e[:, :i], e[:, i:]


def gated(g, u, eg, eu, name):
    """h and its error before its own rounding."""
    a, _ = act(g, name)
    h = a * u
    return h, og.SLOPE * eg * u.abs() + (a.abs() + og.SLOPE * eg) * eu + og.EVAL * h.abs()


def gated_backward(d_h, x, w, name, dtype, saved):
    """(d_x, its tolerance, d_w, its tolerance); arguments in binary64."""
    g, u, eg, eu = project(x, w)
    a, da = act(g, name)
    f = torch.cat([u * da, a], 1)
    e = torch.cat([(da.abs() + eg) * eu + u.abs() * eg + og.EVAL * u.abs() * og.SLOPE * (1 + g.abs()),
                   og.SLOPE * eg + og.EVAL * a.abs()], 1)
    if saved:
        e = e + og.KEPT * (f.abs() + e)
    d = torch.cat([d_h, d_h], 1)
    dgu = d * f
    t = d.abs() * e
    t = t + (og.HALF[dtype] + 2 * og.ADD) * (dgu.abs() + t) + og.TINY[dtype]
    out = []
    for p, pt, q in ((dgu, t, w), (dgu.t(), t.t(), x)):
        v = p @ q
        tol = pt @ q.abs() + (p.shape[1] + 2) * og.ADD * ((p.abs() + pt) @ q.abs())
        out += [v, rounded(v, tol, dtype)]
    return tuple(out)


def w4_product(x, codes, scale, zeros, group):
    """x W^T and its error before its own rounding."""
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1).double()
    s = scale.double().repeat_interleave(group, 1)
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, 1)
    big = x.abs() @ s.abs().t() * 31.0
    return x @ ((q - z) * s).t(), big * (group + scale.shape[1] + 4) * ow.ADD
