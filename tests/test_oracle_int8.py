"""Pins of the int8 oracle: a worked cast, exact rationals, and closed forms."""
from fractions import Fraction

import numpy as np

from oracle import int8


def test_cast_worked_example():
    x = np.zeros((3, 4), np.float32)
    x[0] = [127.0, 0.5, 1.5, -2.5]                   # scale 1: ties go to the even code
    x[1] = [1e-6, -1e-6, 0, 0]                       # below the floor on the row maximum
    q, s = int8.cast(x)
    assert q.tolist() == [[127, 0, 2, -2], [1, -1, 0, 0], [0, 0, 0, 0]]
    assert s[0] == 1.0 and s[1] == s[2] == np.float32(np.float32(1e-4) / np.float32(127))


def test_cast_error_bound():
    x = np.random.default_rng(0).standard_normal((20, 64)).astype(np.float32)
    q, s = int8.cast(x)
    assert np.all(np.abs(q.astype(np.float64) * s[:, None] - x) <= s[:, None] * (0.5 + 1e-5)) and np.abs(q).max() == 127


def test_gemm_against_rationals():
    rng = np.random.default_rng(1)
    qa, qb = rng.integers(-128, 128, (3, 48)).astype(np.int8), rng.integers(-128, 128, (4, 48)).astype(np.int8)
    sa, sb = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32)
    d = int8.gemm_nt(qa, sa, qb, sb)
    for i in range(3):
        for j in range(4):
            total = sum(int(a) * int(b) for a, b in zip(qa[i], qb[j]))
            exact = total * Fraction(float(sa[i])) * Fraction(float(sb[j]))
            assert abs(Fraction(float(d[i, j])) - exact) <= abs(exact) * Fraction(3, 1 << 24)


def test_gemm_closed_forms():
    one = np.ones((2, 256), np.int8)
    s = np.ones(2, np.float32)
    assert np.all(int8.gemm_nt(one, s, one, s) == 256)
    low = np.full((1, 131071), -128, np.int8)        # the longest exact sum
    assert int8.gemm_nt(low, s[:1], low, s[:1])[0, 0] == np.float32(131071 * 16384)
