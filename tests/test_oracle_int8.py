"""The INT8 oracle against exact rationals, closed forms, differences and
planted mistakes."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import int8 as o

F = np.float32


def rng(k):
    return np.random.Generator(np.random.PCG64([41, k]))


def fp32(x):
    """A rational rounded to binary32 (nearest, ties to even), by bisection over
    neighbours; normal range only."""
    f = F(float(x))
    best = min((abs(Fraction(float(c)) - x), int(np.asarray(c).view(np.uint32)) & 1, i, c)
               for i, c in enumerate((np.nextafter(f, F(-np.inf)), f, np.nextafter(f, F(np.inf)))))
    return best[3]


def test_scales_and_codes_against_exact_rationals():
    x = np.concatenate([(rng(0).standard_normal((40, 9)) * 10.0 ** rng(1).integers(-30, 30, (40, 1))).astype(F),
                        np.array([[127, 63.5, 0.5, 1.5, 2.5, -0.5, -1.5, -127, 0]], F)])
    q, s = o.quantize(x)
    for i, row in enumerate(x):
        amax = max(abs(Fraction(float(v))) for v in row)
        assert s[i] == fp32(amax / 127), i
        inv = fp32(1 / Fraction(float(s[i])))
        for v, c in zip(row, q[i]):
            p = Fraction(float(v)) * Fraction(float(inv))
            p = Fraction(0) if p == 0 else Fraction(float(fp32(p))) if abs(p) > Fraction(1, 2 ** 100) else p
            lo = p.numerator // p.denominator
            want = lo if p - lo < Fraction(1, 2) else lo + 1 if p - lo > Fraction(1, 2) else lo + lo % 2
            assert c == want, (i, v)
    assert list(q[-1]) == [127, 64, 0, 2, 2, 0, -2, -127, 0]  # ties to even
    assert np.abs(q).max() == 127


def test_degenerate_rows():
    x = np.zeros((6, 4), F)
    x[1] = [1e-44, -1e-44, 0, 0]
    x[2] = [1, np.inf, 2, 3]
    x[3] = [np.nan, 1, 0, 0]
    x[4] = [F(3.4e38), -F(3.4e38), 1, 0]
    x[5] = 2.0 ** -126
    q, s = o.quantize(x)
    assert s[0] == 1 and not q[0].any()
    assert s[1] == F(2.0 ** -126) and not q[1].any()  # codes of 1e-44 / 2^-126 are 0
    assert np.isnan(s[2]) and np.isnan(s[3]) and not q[2].any() and not q[3].any()
    assert list(q[4]) == [127, -127, 0, 0]
    assert s[5] == F(2.0 ** -126) and (q[5] == 1).all()


def test_dequantized_error_is_half_a_step():
    x = rng(2).standard_normal((50, 33)).astype(F)
    q, s = o.quantize(x)
    err = np.abs(q.astype(np.float64) * s.astype(np.float64)[:, None] - x)
    assert (err <= s[:, None] * (0.5 + 127 * 2.0 ** -22)).all()
    wrong = np.trunc(x / s[:, None])  # planted: cut instead of rounded
    assert not (np.abs(wrong * s[:, None] - x) <= s[:, None] * 0.51).all()


def test_gemm_against_integers():
    a, b = rng(3).integers(-127, 128, (5, 300)).astype(np.int8), rng(4).integers(-127, 128, (7, 300)).astype(np.int8)
    sa, sb = 2.0 ** rng(5).integers(-9, 9, 5), 2.0 ** rng(6).integers(-9, 9, 7)
    c = o.gemm(a, sa, b, sb, bias=np.arange(7))
    for m in range(5):
        for n in range(7):
            t = sum(int(x) * int(y) for x, y in zip(a[m], b[n]))
            assert c[m, n] == t * sa[m] * sb[n] + n
    # the bound holds for a binary32 evaluation and not for one of half the width
    bias = rng(7).standard_normal(7).astype(F)
    sa, sb = rng(8).random(5).astype(F), rng(9).random(7).astype(F)
    c = o.gemm(a, sa, b, sb, bias)
    t = (a.astype(np.int64) @ b.T.astype(np.int64)).astype(F)
    got = (t * sa[:, None]) * sb + bias
    bound = o.gemm_bound(c, bias, 0.0)
    assert (np.abs(got - c) <= bound).all()
    assert not (np.abs(got.astype(np.float16) - c) <= bound).all()


def test_kept_blocks_are_rows_of_their_own():
    gu = rng(10).standard_normal((3, 2 * 300)).astype(F)
    q, s = o.keep(gu)
    assert s.shape == (3, 6)
    for h in range(2):
        for k, (lo, hi) in enumerate(((0, 128), (128, 256), (256, 300))):
            bq, bs = o.quantize(gu[:, h * 300 + lo:h * 300 + hi])
            assert (q[:, h * 300 + lo:h * 300 + hi] == bq).all() and (s[:, 3 * h + k] == bs).all()
    g, u = o.kept(q, s)
    assert np.abs(g - gu[:, :300]).max() <= s.max() * 0.51 and np.abs(u - gu[:, 300:]).max() <= s.max() * 0.51


@pytest.mark.parametrize("g", [-30.0, -3.0, -0.4, 0.0, 0.7, 5.0, 30.0])
def test_gradient_against_differences(g):
    u, da, h = -1.7, 0.3, 1e-5
    dg, du = o.swiglu_bwd(da, g, u)
    assert abs(dg - da * (o.swiglu(g + h, u) - o.swiglu(g - h, u)) / (2 * h)) < 1e-8
    assert abs(du - da * (o.swiglu(g, u + h) - o.swiglu(g, u - h)) / (2 * h)) < 1e-8


def test_activation_values():
    assert o.swiglu(0.0, 3.0) == 0
    assert abs(o.swiglu(1.0, 1.0) - 0.7310585786300049) < 1e-15  # 1 / (1 + 1/e)
    g = rng(11).standard_normal(100) * 5
    assert np.allclose(o.swiglu(g, 1) - o.swiglu(-g, 1), g, atol=1e-14)  # g p + g (1 - p)


def test_bounds_hold_for_binary32_and_not_for_less():
    r = rng(12)
    g, u, da = (r.standard_normal(20000).astype(F) * F(k) for k in (6, 2, 1e-3))
    p = F(1) / (F(1) + np.exp2(g * F(-1.4426950408889634)))
    a = g * p * u
    dg, du = da * u * (p * (F(1) + g * (F(1) - p))), da * (g * p)
    ea, edg, edu = o.swiglu_bounds(da, g, u, 0.0)
    rdg, rdu = o.swiglu_bwd(da, g, u)
    for got, ref, e in ((a, o.swiglu(g, u), ea), (dg, rdg, edg), (du, rdu, edu)):
        assert (np.abs(got - ref) <= e).all()
        assert np.mean(np.abs(o.bf16(got) - ref) <= e) < 0.1
    wrong = da * u * (p * (F(1) + g * p))  # planted: p in the place of 1 - p
    assert np.mean(np.abs(wrong - rdg) <= edg) < 0.1


def test_wgrad():
    r = rng(13)
    dy = r.integers(-8, 9, (37, 5)).astype(np.float64)
    q = r.integers(-127, 128, (37, 6)).astype(np.int8)
    s = 2.0 ** r.integers(-3, 3, 37)
    dw, bound = o.wgrad(dy, q, s)
    for n in range(5):
        for k in range(6):
            assert dw[n, k] == sum(Fraction(float(dy[t, n])) * int(q[t, k]) * Fraction(float(s[t])) for t in range(37))
    # a scale that is no power of two rounds each product to bf16
    dw, bound = o.wgrad(np.ones((1, 1)), np.array([[127]], np.int8), np.array([F(0.1)]))
    assert dw[0, 0] == 12.6875 and (bound > 0).all()  # bf16(12.7)
    assert np.isnan(o.wgrad(np.ones((2, 1)), np.zeros((2, 1), np.int8), np.array([1, np.nan], F))[0]).all()
