"""Plain 64-bit reference of stochastic rounding by 16 bits, one step and whole recurrences (the format and the 7-bit
rounding: _ref8.py)."""
from __future__ import annotations

import numpy as np

import _ref8 as R


def halves(seed: int, step: int, stream: int, n: int, first: int = 0):
    """The 16 bits drawn for each of the elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    pair = i >> np.uint64(1)
    h = R.pcg(seed & R.M32)
    h = R.pcg((seed >> 32) ^ int(h))
    h = R.pcg((step & R.M32) ^ int(h))
    h = R.pcg((stream & R.M32) ^ int(h))
    w = R.pcg((pair & np.uint64(R.M32)) ^ R.pcg((pair >> np.uint64(32)) ^ h))
    return ((w >> (np.uint64(16) * (i & np.uint64(1)))) & np.uint64(0xFFFF)).astype(np.float64)


def grid16(y: np.ndarray, h: np.ndarray) -> np.ndarray:
    """Roots over their scale (>= 0) on the e4m3 grid: floor(y / u + (h + 1/2) / 65536) u, above zero at least 2^-9."""
    y = np.where(y > 0, np.clip(y, 2.0 ** -9, 448.0), 0.0)
    u = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    return np.floor(y / u + (h + 0.5) / 65536) * u


def swapped(h: np.ndarray) -> np.ndarray:
    """The two bytes of each half exchanged: what rounds exp_avg."""
    h = h.astype(np.uint64)
    return ((h >> np.uint64(8)) | ((h & np.uint64(255)) << np.uint64(8))).astype(np.float64)


def signed16(x: np.ndarray, h: np.ndarray) -> np.ndarray:
    """exp_avg over its scale on the e4m3 grid: floor(|x| / u + (h + 1/2) / 65536) u under x's sign."""
    a = np.minimum(np.abs(x), 448.0)
    u = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.floor(a / u + (h + 0.5) / 65536) * u, x)


def check_exp_avg16(codes, scales, value, bound, h, name="exp_avg"):
    """The stored codes and scales are what `value`, known to +- bound, rounds to with the (exchanged) draws h."""
    n = len(codes)
    amax, err = np.abs(R.rows(value)), R.rows(bound)
    lo, hi = R.scale_of(np.maximum(amax - err, 0).max(1)), R.scale_of((amax + err).max(1))
    s = scales.astype(np.float64)
    assert ((lo <= s) & (s <= hi)).all(), f"{name}: scales"
    per = np.repeat(s, R.BLOCK)[:n]
    a, b = (signed16(np.maximum(np.abs(value) + k * bound, 0) / per, h) for k in (-1, 1))
    got = R.TABLE[codes]
    side = (np.abs(value) <= bound) | (got == 0) | (np.sign(got) == np.sign(value))
    bad = ~(side & (a <= np.abs(got)) & (np.abs(got) <= b))
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {n} codes", value[bad][:3], got[bad][:3], a[bad][:3], b[bad][:3])


def check_root16(codes, scales, value, bound, h, name="root"):
    """The stored codes and scales are what `value` (>= 0), known to +- bound, rounds to with the draws h."""
    n = len(codes)
    amax, err = R.rows(value), R.rows(bound)
    lo, hi = R.scale_of(np.maximum(amax - err, 0).max(1)), R.scale_of((amax + err).max(1))
    s = scales.astype(np.float64)
    assert ((lo <= s) & (s <= hi)).all(), f"{name}: scales"
    per = np.repeat(s, R.BLOCK)[:n]
    a = grid16(np.maximum(value - bound, 0) / per, h)
    a = np.where(value > 0, np.maximum(a, 2.0 ** -9), a)
    b = grid16((value + bound) / per, h)
    b = np.where(value > 0, b, 0.0)
    got = R.TABLE[codes]
    bad = ~((a <= got) & (got <= b))
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {n} codes", value[bad][:3], got[bad][:3], a[bad][:3], b[bad][:3])


def grads(kind: str, step: int, n: int) -> np.ndarray:
    """The grads of a long run, binary32 values: normal ones or ones that do not change."""
    if kind == "constant":
        return np.linspace(0.5, 2.0, n).astype(np.float32)
    return np.random.default_rng(1000 + step).normal(size=n).astype(np.float32)


def follow(steps: int, b2: float, kind: str, n: int, seed: int):
    """exp_avg_sq after a run from zero: (the exact one, the one whose root is stored with 16-bit rounding)."""
    v, r = np.zeros(n), np.zeros(n)
    for t in range(1, steps + 1):
        g2 = grads(kind, t, n).astype(np.float64) ** 2
        v = b2 * v + (1 - b2) * g2
        x = np.sqrt(b2 * r * r + (1 - b2) * g2)
        s = np.repeat(R.scale_of(R.rows(x).max(1)), R.BLOCK)[:n]
        r = grid16(x / s, halves(seed, t, 0, n)) * s
    return v, r * r


def follow_exp_avg(steps: int, b1: float, n: int, seed: int):
    """exp_avg after a run from zero, grads of mean 1: (the exact one, the one stored with 16-bit rounding)."""
    e, m = np.zeros(n), np.zeros(n)
    for t in range(1, steps + 1):
        g = 1.0 + grads("normal", t, n).astype(np.float64)
        e = b1 * e + (1 - b1) * g
        x = b1 * m + (1 - b1) * g
        s = np.repeat(R.scale_of(np.abs(R.rows(x)).max(1)), R.BLOCK)[:n]
        m = signed16(x / s, swapped(halves(seed, t, 0, n))) * s
    return e, m


def run_bounds(b2: float):
    """The mean of a followed exp_avg_sq over the exact one.  Rounding x to the grid's neighbours keeps x's mean and adds
    u^2 f (1 - f) to x^2's, f u the distance to one of them: with f u the step's own move, (1 - beta2) |g^2 / v - 1| x / 2,
    at most (u / x) |g^2 / v - 1| / 2 of v in all, u / x <= 1/8.  |g^2 / v - 1| has the mean 0.97 for normal grads; from
    zero and with grads that do not change it falls from where the run begins: below 1.  The mean over the elements is
    known to 2 %.  The 7 bits (beta2 up to 0.99) take up to u / 256 off a root at each step, 1 / 1024 off exp_avg_sq,
    which adds up to 1 / 1024 / (1 - beta2) of it."""
    return 0.98 - (1.0 / 1024 / (1 - b2) if b2 <= 0.99 else 0.0), 1.02 + 1.0 / 16
