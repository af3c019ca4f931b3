"""How far the roots and coefficients of the norms' results are off, from their steps in exact arithmetic.

u = 2^-24.  root(): the binary32 root of a rounded sum is 1.5 u off, 0.5 / y rounded by u, so the first step leaves
1.5^2 / 2 u^2 + 1.5 u^2 = 2.625 u^2, the second 2.625 u^2 x 2.5 u and the rounding of the last addition, 2^-53.  tensor_norm():
residual and quotient rounded by u each, 1.125 u^2 + 2 u x 1.5 u = 4.125 u^2 before the last rounding.  clip_coefficient(): the
first quotient 3 u, then residual, d and quotient u each: 9 u^2.  All to the first order: another 2 % for the rest."""
from fractions import Fraction as Fr

import numpy as np
import pytest

U = Fr(1, 1 << 24)
DRAWS = 4000


def f32(x):
    """A binary64 number to the nearest binary32."""
    return Fr(float(np.float32(x)))


def round32(x):
    """A fraction in the normal range to 24 bits, half to even."""
    if x == 0:
        return x
    e = 0
    y = abs(x)
    while y >= 1 << 24:
        y, e = y / 2, e + 1
    while y < 1 << 23:
        y, e = y * 2, e - 1
    r = Fr(round(y)) * Fr(2) ** e
    return r if x > 0 else -r


def round64(x):
    return Fr(float(x))


def root32(f):
    """The binary32 root of a binary32 value: of a binary64 root, which is near no tie (a tie's square has 50 bits)."""
    return round32(Fr(float(np.sqrt(np.float64(float(f))))))


def exact_root(s):
    """A root to 2^-90."""
    y = Fr(float(np.sqrt(np.float64(float(s)))))
    for _ in range(2):
        y = (y + s / y) / 2
        y = Fr(round(y * (1 << 200)), 1 << 200)
    return y


@pytest.fixture(scope="module")
def draws():
    rng = np.random.default_rng(3)
    return [(Fr(float(a)), Fr(float(b))) for a, b in zip(rng.uniform(1.0, 4.0, DRAWS), rng.uniform(1.0, 2.0, DRAWS))]


def test_roots(draws):
    first, last, norm = Fr(0), Fr(0), Fr(0)
    for s, _ in draws:
        want = exact_root(s)
        y0 = root32(f32(float(s)))
        half = round32(Fr(1, 2) / y0)
        y = y0
        for k in range(2):
            r = round64(s - y * y)  # fma: rounded once
            y = round64(y + r * half)
            if k == 0:
                first = max(first, abs(y / want - 1))
        last = max(last, abs(y / want - 1))
        rest = round32(round64(s - y0 * y0))
        norm = max(norm, abs((y0 + round32(rest / (2 * y0))) / want - 1))
    assert first <= Fr(102, 100) * Fr(2625, 1000) * U * U + Fr(1, 1 << 53)
    assert last <= Fr(1, 1 << 53) * (1 + Fr(1, 1 << 15))
    assert norm <= Fr(102, 100) * Fr(4125, 1000) * U * U
    assert norm / U <= Fr(1, 1 << 21)  # beside the last rounding's u


def test_coefficients(draws):
    worst = Fr(0)
    for d, limit in draws:
        d, limit = (d, limit) if limit < d else (limit, d)
        if limit == d:
            continue
        fd, fl = f32(float(d)), f32(float(limit))
        q = round32(fl / fd)
        rest = round32(round64(limit - q * d))
        worst = max(worst, abs((q + round32(rest / fd)) / (limit / d) - 1))
    assert worst <= Fr(102, 100) * 9 * U * U and worst / U <= Fr(1, 1 << 20)
    assert worst > 2 * U * U  # it is not the u^2 / 2 of exact factors
