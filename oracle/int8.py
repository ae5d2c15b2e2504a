"""INT8 recipe: symmetric codes with one scale for each row, column or block of
128, the products of such codes, and the gated activation whose input is kept
in them (test infrastructure).

Definitions (binary32 where a value is called fp32, 64 bits or exact integers
elsewhere):
    s     = max(fp32(amax / 127), 2^-126); 1 for amax 0; NaN for one not finite
    code  = rint(fp32(v fp32(1 / s))), nearest, ties to even; 0 where s is NaN
    C     = (sum_k A B) sa sb + bias
    x'    = bf16(fp32(code s)),  dW[n, k] = sum_t dY[t, n] x'[t, k]
    a     = g p u,  p = 1 / (1 + exp(-g))
    dg    = da u p (1 + g (1 - p)),  du = da g p   with g, u = fp32(code s)
"""

import numpy as np

F = np.float32
U = 2.0 ** -24  # half a step of binary32
TINY = F(2.0 ** -126)
BLOCK = 128


def scale(amax):
    """Scales of an array of binary32 maxima."""
    amax = np.asarray(amax, F)
    with np.errstate(all="ignore"):
        s = np.maximum(amax / F(127), TINY)
    s = np.where(amax == 0, F(1), s)
    return np.where(np.isfinite(amax), s, F("nan")).astype(F)


def codes(v, s):
    """Codes of binary32 values under scales of a broadcast shape."""
    with np.errstate(all="ignore"):
        p = np.asarray(v, F) * (F(1) / np.asarray(s, F))
        c = np.rint(p)
    return np.where(np.isnan(s), 0, np.nan_to_num(c, nan=0.0, posinf=0.0, neginf=0.0)).astype(np.int8)


def amax(x, axis):
    with np.errstate(all="ignore"):
        a = np.abs(np.asarray(x, F))
    if a.shape[axis] == 0:
        return np.zeros([n for i, n in enumerate(a.shape) if i != axis], F)
    return a.max(axis=axis)  # a NaN among them gives NaN


def quantize(x):
    """(codes, scales) of the rows."""
    s = scale(amax(x, 1))
    return codes(x, s[:, None]), s


def gemm(a, sa, b, sb, bias=None):
    """C in 64 bits from exact sums."""
    total = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T  # exact below 2^53
    c = total * np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)
    return c if bias is None else c + np.asarray(bias, np.float64)


def gemm_bound(c, bias, half_step):
    """How far a C that is scaled in binary32 and rounded once may be: the
    conversion of the sum and two products round once each (3 u of their
    result, a fourth for second order), the addition and the output once."""
    c = np.abs(c)
    p = c if bias is None else c + np.abs(np.asarray(bias, np.float64))
    e = 4 * U * p + U * c
    return e + half_step * (c + e) + 2.0 ** -133


def blocks(cols):
    return -(-cols // BLOCK)


def keep(gu):
    """(codes, scales) of g and u in blocks along the row."""
    gu = np.asarray(gu, F)
    C = gu.shape[1] // 2
    q = np.zeros(gu.shape, np.int8)
    s = np.ones((gu.shape[0], 2 * blocks(C)), F)
    for half in range(2):
        for k in range(blocks(C)):
            lo, hi = half * C + k * BLOCK, half * C + min(C, (k + 1) * BLOCK)
            q[:, lo:hi], s[:, half * blocks(C) + k] = quantize(gu[:, lo:hi])
    return q, s


def kept(q, s):
    """g and u that kept codes stand for, binary32."""
    C = q.shape[1] // 2
    nb = blocks(C)
    at = np.arange(C) // BLOCK
    with np.errstate(all="ignore"):
        g = q[:, :C].astype(F) * s[:, :nb][:, at]
        u = q[:, C:].astype(F) * s[:, nb:][:, at]
    return g, u


def sigmoid(g):
    g = np.asarray(g, np.float64)
    with np.errstate(all="ignore"):
        return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def swiglu(g, u):
    return np.asarray(g, np.float64) * sigmoid(g) * np.asarray(u, np.float64)


def swiglu_bwd(da, g, u):
    da, g, u = (np.asarray(v, np.float64) for v in (da, g, u))
    p = sigmoid(g)
    return da * u * p * (1 + g * (1 - p)), da * g * p


def sigmoid_error(g, p):
    """Error of p in binary32 from a base-2 exponential and a reciprocal that
    are off by one step each: the argument -g log2(e) carries two roundings,
    2 u |g| of the exponential, whose own step is 2 u; (1 - p) of that reaches
    p; the sum 1 + exp rounds by u and the reciprocal by 2 u.  Below 2^-126 an
    exponential or a p may be taken for 0."""
    return p * (2 * (np.abs(g) + 1) * (1 - p) + 3) * U + 2.0 ** -125


def sigmoid_error_f32(g, p):
    """The same of what fp32 data take: the exponent's fraction, at most a half,
    carries two roundings of 2^-25, 0.7 u of the exponential, whose own step is
    2 u; (1 - p) of that reaches p; the sum and the division round by u.  Where
    1 + exp is not finite, p is taken for 0."""
    return p * (2.7 * (1 - p) + 2) * U + 2.0 ** -128


def swiglu_bounds(da, g, u, half_step, error=sigmoid_error):
    """Bounds of (a, dg, du) against swiglu and swiglu_bwd; da may be None (a
    alone); error is that of p."""
    g, u = np.asarray(g, np.float64), np.asarray(u, np.float64)
    p = sigmoid(g)
    dp = error(g, p)
    floor = 2.0 ** -126

    def out(value, err):
        err = 1.01 * err
        return err + half_step * (np.abs(value) + err) + floor

    a = g * p * u
    ea = out(a, np.abs(g * u) * (dp + 3 * U * p))
    if da is None:
        return ea, None, None
    da = np.asarray(da, np.float64)
    t = 1 + g * (1 - p)
    et = np.abs(g) * (dp + U + 2 * U * (1 - p)) + 2 * U * np.abs(t)
    dg, du = da * u * p * t, da * g * p
    edg = out(dg, np.abs(da * u) * (p * et + np.abs(t) * dp + 4 * U * np.abs(p * t)))
    edu = out(du, np.abs(da * g) * (dp + 3 * U * p))
    return ea, edg, edu


def bf16(x):
    """binary32 values rounded to bfloat16 (nearest, ties to even), as binary32; NaN stays NaN."""
    x = np.ascontiguousarray(x, F)
    b = x.view(np.uint32)
    r = ((b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(F)
    return np.where(np.isnan(x), x, r)


def wgrad(dy, q, s):
    """(dW, bound): dW in 64 bits, and how far a binary32 sum of the exact
    products may be, in any order and with partial sums that are cut instead of
    rounded (2 u each)."""
    with np.errstate(all="ignore"):
        x = bf16(np.asarray(q).astype(F) * np.asarray(s, F)[:, None]).astype(np.float64)
    dy = np.asarray(dy, np.float64)
    return dy.T @ x, 2 * U * (len(dy) + 16) * (np.abs(dy).T @ np.abs(x))
