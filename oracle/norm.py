"""Residual addition, RMS norm, its gradient, and the global gradient norm with
clipping, in 64 bits (test infrastructure).

Definitions (one row x of C elements, weight g):
    h    = x + r                     rounded to the data type by the caller
    rstd = (sum h^2 / C + eps)^(-1/2)
    y    = h rstd g
Gradient of sum(dy y) + sum(dres h) with respect to x (and r):
    dx   = rstd (dy g - n mean(dy g n)) + dres,   n = h rstd
    dg   = sum over rows of dy n
Clipping: out = t min(1, max_norm / (norm + 1e-6)), norm the square root of
the sum of squares over all tensors.

The FP8 copies of y are those of the recipes module: ``normed_f32`` restates
the two binary32 products, so that codes can be compared bit for bit.
"""

import math

import numpy as np


def rstd(h, eps):
    h = np.asarray(h, dtype=np.float64)
    return 1.0 / np.sqrt((h * h).sum(axis=1) / h.shape[1] + eps)


def normed(h, r, g):
    """y in 64 bits from a given rstd."""
    return np.asarray(h, np.float64) * np.asarray(r, np.float64)[:, None] * np.asarray(g, np.float64)


def normed_f32(h, r, g):
    """y as binary32: fp32(fp32(h rstd) gamma), each product rounded once."""
    f = np.float32
    with np.errstate(all="ignore"):
        return (np.asarray(h, f) * np.asarray(r, f)[:, None]) * np.asarray(g, f)


def norm_bwd(dy, h, r, g, dres=None):
    """(dx, dgamma) in 64 bits from a given rstd."""
    dy, h, g = (np.asarray(v, np.float64) for v in (dy, h, g))
    r = np.asarray(r, np.float64)[:, None]
    n, dn = h * r, dy * g
    dx = r * (dn - n * (dn * n).sum(axis=1, keepdims=True) / h.shape[1])
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * n).sum(axis=0)


def norm_bwd_bound(dy, h, r, g, dres, longest, half_step):
    """How far a binary32 dx may be from norm_bwd's, element by element, when no
    sum of a row is a chain of more than ``longest`` additions and the result
    is rounded once with a relative error of half_step.

    With u = 2^-24: dn and n carry one rounding each; n m - dn, the product by
    rstd and the addition of dres one each; m carries its own sum's error,
    (longest + 3) u mean|dn n|; one more u per term covers second order."""
    u = 2.0 ** -24
    dy, h, g = (np.asarray(v, np.float64) for v in (dy, h, g))
    r = np.asarray(r, np.float64)[:, None]
    n, dn = h * r, dy * g
    m = (dn * n).sum(axis=1, keepdims=True) / h.shape[1]
    mabs = np.abs(dn * n).sum(axis=1, keepdims=True) / h.shape[1]
    b = np.abs(r) * (5 * np.abs(dn) + 5 * np.abs(n * m) + (longest + 4) * np.abs(n) * mabs)
    ref = r * (dn - n * m)
    if dres is not None:
        b = b + 2 * np.abs(dres)
        ref = ref + np.asarray(dres, np.float64)
    b = u * b
    return b + half_step * (np.abs(ref) + b)


def clip(tensors, max_norm):
    """(outs, sum of squares, norm) in 64 bits."""
    s = math.fsum(float(np.dot(t.ravel(), t.ravel())) for t in (np.asarray(t, np.float64) for t in tensors))
    norm = math.sqrt(s)
    k = min(1.0, max_norm / (norm + 1e-6))
    return [np.asarray(t, np.float64) * k for t in tensors], s, norm
