"""Pins of the int8 oracle: hand-worked rows, exact fractions, and the bounds that
the GPU tests rest on."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8 as o8


def test_hand_worked_row():
    # amax 127 gives the scale fl(127 * fl(1/127)), which is 1 exactly.
    y = np.array([[127.0, -127.0, 0.5, 1.5, -2.5, 63.49, 0.0, -0.0]], dtype=np.float32)
    q, s = o8.row_codes(y)
    assert s[0] == 1.0
    assert q[0].tolist() == [127, -127, 0, 2, -2, 63, 0, 0]


def test_zero_and_tiny_rows_keep_the_smallest_scale():
    y = np.array([[0.0, -0.0], [1e-45, 0.0], [2.0 ** -126 * 3, -2.0 ** -126 * 5]], dtype=np.float32)
    q, s = o8.row_codes(y)
    assert (s == np.float32(2.0 ** -126)).all()
    assert q.tolist() == [[0, 0], [0, 0], [3, -5]]


def test_rows_that_are_not_finite():
    y = np.array([[1.0, np.inf], [np.nan, 2.0], [-np.inf, np.nan], [1.0, 2.0]], dtype=np.float32)
    q, s = o8.row_codes(y)
    assert np.isnan(s[:3]).all() and not np.isnan(s[3]) and (q[:3] == 0).all()


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_codes_stay_inside_127_and_near_the_exact_quotient(seed):
    """s is within 1.5 * 2^-24 * 2 of amax/127 and r, y*r add 2^-24 each: |y*r - 127 y/amax| <= 127 * 5 * 2^-24."""
    g = np.random.default_rng(seed)
    y = (g.standard_normal((200, 48)) * 10.0 ** g.uniform(-30, 30, (200, 1))).astype(np.float32)
    q, s = o8.row_codes(y)
    for i in range(200):
        amax = Fraction(float(np.max(np.abs(y[i]))))
        assert max(abs(int(v)) for v in q[i]) == 127
        for v, c in zip(y[i], q[i]):
            exact = Fraction(float(v)) * 127 / amax
            assert abs(exact - int(c)) <= Fraction(1, 2) + Fraction(127 * 5, 2 ** 24)


def test_rmsnorm_against_fractions():
    g = np.random.default_rng(5)
    x = o8.round_to(g.standard_normal((3, 32)), "bf16")
    r = o8.round_to(g.standard_normal((3, 32)), "bf16")
    w = o8.round_to(1 + 0.1 * g.standard_normal(32), "bf16")
    y, h = o8.rmsnorm(x, w, 2.0 ** -20, "bf16", residual=r)
    for i in range(3):
        ms = sum(Fraction(float(v)) ** 2 for v in h[i]) / 32 + Fraction(1, 2 ** 20)
        for k in range(32):
            # inv 2^-24 (and the float64 steps), the products 2^-24 each
            want = float(h[i, k]) / float(ms) ** 0.5 * float(w[k])
            assert abs(float(y[i, k]) - want) <= abs(want) * (3 * 2.0 ** -24 + 2.0 ** -40)
            total = float(x[i, k]) + float(r[i, k])
            assert abs(float(h[i, k]) - total) <= 2.0 ** -8 * abs(total) + 2.0 ** -134


def test_gemm_against_fractions():
    g = np.random.default_rng(6)
    aq, bq = g.integers(-128, 128, (3, 16)).astype(np.int8), g.integers(-128, 128, (4, 16)).astype(np.int8)
    a_s, b_s = g.random(3).astype(np.float32), g.random(4).astype(np.float32)
    c = o8.gemm(aq, a_s, bq, b_s)
    for m in range(3):
        for n in range(4):
            acc = sum(int(a) * int(b) for a, b in zip(aq[m], bq[n]))
            want = acc * Fraction(float(a_s[m])) * Fraction(float(b_s[n]))
            assert abs(Fraction(float(c[m, n])) - want) <= abs(want) * Fraction(4, 2 ** 24)
    assert np.allclose(o8.gemm_f64(aq, a_s, bq, b_s), c, rtol=2.0 ** -21, atol=0)
