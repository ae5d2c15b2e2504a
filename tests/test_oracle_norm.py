"""Pins of the norm and clipping oracle: a plain loop in exact rationals, the
gradient against central differences, closed forms, and the error bound
against a binary32 evaluation (with planted mistakes that it has to catch)."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import norm


def rng(k):
    return np.random.default_rng(k)


def test_rstd_and_y_against_a_loop():
    g = rng(1)
    h, w = g.standard_normal((5, 13)), g.standard_normal(13)
    r = norm.rstd(h, 1e-3)
    y = norm.normed(h, r, w)
    for i in range(5):
        ms = sum(Fraction(float(v)) ** 2 for v in h[i]) / 13
        want = 1 / math.sqrt(float(ms) + 1e-3)
        assert abs(r[i] - want) <= 4e-16 * want
        for c in range(13):
            assert y[i, c] == pytest.approx(h[i, c] * want * w[c], rel=1e-14)


def test_closed_forms():
    # a constant row has an rms of its value
    assert norm.rstd(np.full((1, 7), -4.0), 0.0)[0] == 0.25
    assert norm.rstd(np.zeros((1, 3)), 0.25)[0] == 2.0
    # y does not depend on the scale of h without eps
    h = rng(2).standard_normal((3, 9))
    w = np.ones(9)
    assert np.allclose(norm.normed(h, norm.rstd(h, 0.0), w), norm.normed(8 * h, norm.rstd(8 * h, 0.0), w), rtol=1e-15)


def test_normed_f32_rounds_each_product():
    h, r, w = np.float32([[3.1]]), np.float32([0.7]), np.float32([1.3])
    a = np.float32(np.float64(h[0, 0]) * np.float64(r[0]))
    assert norm.normed_f32(h, r, w)[0, 0] == np.float32(np.float64(a) * np.float64(w[0]))


@pytest.mark.parametrize("with_dres", [False, True])
def test_gradient_against_central_differences(with_dres):
    g = rng(3)
    R, C, eps = 4, 11, 1e-2
    h, w, dy = g.standard_normal((R, C)), g.standard_normal(C), g.standard_normal((R, C))
    dres = g.standard_normal((R, C)) if with_dres else None

    def loss(h, w):
        v = (dy * norm.normed(h, norm.rstd(h, eps), w)).sum()
        return v + (dres * h).sum() if with_dres else v

    dx, dw = norm.norm_bwd(dy, h, norm.rstd(h, eps), w, dres)
    d = 1e-5
    for i in range(R):
        for c in range(C):
            e = np.zeros((R, C))
            e[i, c] = d
            assert (loss(h + e, w) - loss(h - e, w)) / (2 * d) == pytest.approx(dx[i, c], abs=1e-7)
    for c in range(C):
        e = np.zeros(C)
        e[c] = d
        assert (loss(h, w + e) - loss(h, w - e)) / (2 * d) == pytest.approx(dw[c], abs=1e-7)


def test_bound_holds_for_binary32_and_catches_mistakes():
    g = rng(4)
    f = np.float32
    R, C = 16, 200
    h, w, dy, dres = (g.standard_normal(s).astype(f) for s in ((R, C), C, (R, C), (R, C)))
    r = norm.rstd(h, 1e-5).astype(f)
    ref, _ = norm.norm_bwd(dy, h, r, w, dres)
    bound = norm.norm_bwd_bound(dy, h, r, w, dres, C, 0.0)
    n, dn = h * r[:, None], dy * w

    def f32_dx(m):
        return r[:, None] * (dn - n * m) + dres

    m = (np.cumsum(dn * n, axis=1, dtype=f)[:, -1:] / f(C)).astype(f)
    assert (np.abs(f32_dx(m) - ref) <= bound).all()
    # planted: a row's mean over one element less, a lost residual gradient
    assert not (np.abs(f32_dx(m * f(C / (C - 1.0))) - ref) <= bound).all()
    assert not (np.abs(f32_dx(m) - dres - ref) <= bound).all()


def test_clip():
    a, b = np.array([3.0, 0.0]), np.array([[4.0]])
    outs, s, n = norm.clip([a, b], 1.0)
    assert (s, n) == (25.0, 5.0)
    assert np.allclose(outs[0], a / 5, rtol=1e-6) and np.allclose(outs[1], b / 5, rtol=1e-6)
    outs, _, _ = norm.clip([a, b], 10.0)
    assert (outs[0] == a).all() and (outs[1] == b).all()
    assert norm.clip([], 1.0)[1:] == (0.0, 0.0)
