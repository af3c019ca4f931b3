"""The update's square root without a GPU: one Newton step in binary32 from any reciprocal root of the hardware's accuracy."""
import numpy as np
import pytest


def newton(v, y):
    """g = v y; g + (v - g^2) y / 2, each operation rounded to binary32 once (products of two are exact in binary64)."""
    g = (v.astype(np.float64) * y).astype(np.float32)
    rest = (g.astype(np.float64) * g - v).astype(np.float32)
    return (rest.astype(np.longdouble) * (-0.5 * y.astype(np.float64)) + g).astype(np.float32)


@pytest.mark.parametrize("first", [0, 1])
def test_one_newton_step_rounds_correctly_but_for_one_in_a_million(first):
    # every binary32 number of two octaves; errors of the reciprocal root up to 2^-22, the worst at both ends among them
    wrong = 0
    rng = np.random.default_rng(first)
    for a in range(0, 1 << 23, 1 << 20):
        v = ((127 + first) << 23 | np.arange(a, a + (1 << 20), dtype=np.int64)).astype(np.int32).view(np.float32)
        true = np.sqrt(v.astype(np.float64))
        for off in (-1.0, 1.0, rng.uniform(-1, 1, v.size)):
            y = (1.0 / true * (1 + off * 2.0 ** -22)).astype(np.float32)
            r, want = newton(v, y), true.astype(np.float32)
            assert (np.abs(r.view(np.int32) - want.view(np.int32)) <= 1).all()
            wrong += int((r != want).sum())
    assert wrong <= 3 * (1 << 23) * 2e-6
