"""Plain numpy forms of the operators between message and attention, shared by
their tests.  Nothing here uses the package.

Error bounds (derived, not fitted).  u is the output type's unit roundoff.

rows     every step of a code is one rounding in fp32, so codes and the
         residual's sum are held to equality.
norm     the squares are positive, each rounded once, and added in any order by
         at least 32 lanes: the sum is off by at most (cols / 32 + 64) 2^-24 of
         itself, the inverse root by half of that; division, root and products
         add at most 8 2^-24.
product  integer sums below 2^24 are exact in any order, and then the two
         products with the scales, one rounding each, and the output's rounding
         are fixed: held to equality.  Otherwise a sum of K products in any
         order of tensor-core steps errs by at most (K / 8 + 64) 2^-23 sum |x w|.
rope     the angle's half turns are a 24-bit number (off by 2^-24 pi of a half
         turn, 2^-22.3 radians, and 2^-32 turns for the bits cut off), sine and
         cosine by another 2^-22 with the factor, the two products and their sum
         by 3 2^-24: 2^-20 (|a| + |b|) |factor| covers them.  The table's
         frequency is rounded to 2^-52 of itself.
"""
from __future__ import annotations

import numpy as np

U_OUT = {0: 2.0 ** -11, 1: 2.0 ** -8}
TINY = {0: 2.0 ** -25, 1: 2.0 ** -134}  # half of the smallest subnormal


def rows8(v):
    """(codes, A / 127) of fp32 rows, float32 step by step."""
    v = v.astype(np.float32)
    most = np.abs(v).max(1)
    with np.errstate(divide="ignore", over="ignore"):
        f = np.float32(127) / most
    f = np.where(np.isfinite(f), f, np.float32(0))
    return np.rint(v * f[:, None]).astype(np.int8), most / np.float32(127)


def norm_slack(cols):
    return ((cols / 32 + 64) / 2 + 8) * 2.0 ** -24


def rope(x, angle, layout, rot, factor):
    """(values, |a| + |b| of each) in float64; angle [tokens, rot / 2]."""
    x = x.astype(np.float64)
    out, size = x.copy(), np.zeros_like(x)
    at = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., at[0]], x[..., at[1]]
    c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
    out[..., at[0]], out[..., at[1]] = a * c - b * s, b * c + a * s
    size[..., at[0]] = size[..., at[1]] = (np.abs(a) + np.abs(b)) * abs(factor)
    return out, size
