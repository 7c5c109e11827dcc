"""4-bit weights with a scale and a zero point per group, in binary64 (test oracle).

Test infrastructure: see the package docstring for who may import this.

    W[n,k] = (q - z) s;  s = T(fl32(fl32(hi - lo) / 15)), z = clamp(rint(-lo / s), 0, 15)
    (without zero points s = T(fl32(max |w| / 7)), z = 8), q = clamp(rint(w / s) + z, 0, 15);
    s = 0, infinite or NaN: q = z, with zero points z = 0
"""
from __future__ import annotations

import numpy as np

ADD = 2.0 ** -23


def to_type(v, dtype):
    """fp32 values to the 16-bit type, nearest even; as binary64."""
    v = np.asarray(v, np.float32)
    if dtype == "float16":
        return v.astype(np.float16).astype(np.float64)
    u = v.view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def quant(w, group, zeros, dtype):
    """w [N,K] (values of the type, binary64) -> q [N,K], s, z [N,K/group]."""
    n, k = w.shape
    v = w.reshape(n, k // group, group)
    if zeros:
        lo, hi = np.minimum(v.min(2), 0), np.maximum(v.max(2), 0)
        with np.errstate(over="ignore"):
            s = to_type(((hi - lo).astype(np.float32) / np.float32(15)), dtype)
    else:
        s = to_type(np.abs(v).max(2).astype(np.float32) / np.float32(7), dtype)
    ok = (s > 0) & (s < np.inf)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.clip(np.rint(np.where(ok, -lo / s, 0)), 0, 15) if zeros else np.full(s.shape, 8.0)
        r = np.rint(np.where(ok[:, :, None], v / s[:, :, None], 0))
    q = np.clip(r + z[:, :, None], 0, 15).reshape(n, k).astype(np.uint8)
    return q, s, z.astype(np.uint8)


def pack(q):
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    q = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    return q


def values(codes, s, z, group):
    """W in binary64, unrounded; z None: 8."""
    q = unpack(codes).astype(np.float64)
    off = 8.0 if z is None else np.repeat(z.astype(np.float64), group, 1)
    return (q - off) * np.repeat(s, group, 1)


def product(x, codes, s, z, group):
    """x W^T and the error allowed before its own rounding: fp32 sums in any order,
    of products with the codes less any bias up to 16 within a group, each group's
    then multiplied by its scale."""
    y = x @ values(codes, s, z, group).T
    big = np.abs(x) @ np.repeat(np.abs(s), group, 1).T * 31.0
    return y, big * (group + s.shape[1] + 4) * ADD
