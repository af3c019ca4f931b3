"""Plain 64-bit implementation of the 8-bit AdamW step, with the bounds its binary32 kernels must keep.

The formulas are written out in numpy float64; beside each value goes the most
that a binary32 evaluation in the documented order can be off (EPS = 2^-24 per
rounded operation or constant, first order, x 1.1 for the rest).  A stored code
is then checked by monotonicity: rounding the exact value minus and plus that
bound must enclose the stored value.
"""
from __future__ import annotations

import math

import numpy as np

EPS = 2.0 ** -24
TINY = 2.0 ** -140  # binary32 subnormals' spacing and a little
BLOCK = 256
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------- format
def decode_table() -> np.ndarray:
    """The 256 e4m3 values (1 sign, 4 exponent bits of bias 7, 3 fraction bits; no infinities, 0x7f NaN)."""
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            x = math.nan
        out[c] = -x if c & 128 else x
    return out


TABLE = decode_table()


def rows(x: np.ndarray, fill=0) -> np.ndarray:
    """1-D values as rows of one block, the last one filled."""
    n = len(x)
    out = np.full(-(-n // BLOCK) * BLOCK, fill, dtype=x.dtype)
    out[:n] = x
    return out.reshape(-1, BLOCK)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What codes (uint8) and block scales stand for, float64."""
    return (rows(TABLE[codes]) * scales.astype(np.float64)[:, None]).reshape(-1)[:len(codes)]


def scale_of(amax: np.ndarray) -> np.ndarray:
    """The least power of two >= 2^-126 with amax <= 448 S; NaN from 2^126 on."""
    s = np.full(amax.shape, 2.0 ** -126)
    ok = (amax > 0) & (amax < 2.0 ** 126)
    s[ok] = np.maximum(2.0 ** np.ceil(np.log2(amax[ok] / 448.0)), 2.0 ** -126)
    # log2 may miss an exact power by an ulp
    s[ok] = np.where(amax[ok] > 448.0 * s[ok], 2 * s[ok], s[ok])
    s[ok] = np.where((amax[ok] <= 224.0 * s[ok]) & (s[ok] > 2.0 ** -126), s[ok] / 2, s[ok])
    s[~(amax < 2.0 ** 126)] = np.nan
    return s


def grid(x: np.ndarray, k=None) -> np.ndarray:
    """x (|x| <= 448 or a little more) on the e4m3 grid: to nearest even, or with 7 random bits k."""
    a = np.minimum(np.abs(x), 448.0)
    u = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    q = np.rint(a / u) if k is None else np.floor((np.floor(128.0 * a / u) + k) / 128.0)
    return np.copysign(q * u, x)


# ------------------------------------------------------------------- draws
def pcg(x):
    """O'Neill's RXS-M-XS 32-bit permutation."""
    x = np.asarray(x, np.uint64)
    x = (x * np.uint64(747796405) + np.uint64(2891336453)) & np.uint64(M32)
    x = ((x >> ((x >> np.uint64(28)) + np.uint64(4))) ^ x) * np.uint64(277803737) & np.uint64(M32)
    return (x >> np.uint64(22)) ^ x


def draws(seed: int, step: int, stream: int, n: int, first: int = 0):
    """The 7-bit numbers (for exp_avg, for the root) of elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    pair = i >> np.uint64(1)
    h = pcg(seed & M32)
    h = pcg((seed >> 32) ^ int(h))
    h = pcg((step & M32) ^ int(h))
    h = pcg((stream & M32) ^ int(h))
    h = pcg((pair >> np.uint64(32)) ^ h)
    w = pcg((pair & np.uint64(M32)) ^ h)
    half = (w >> (np.uint64(16) * (i & np.uint64(1)))) & np.uint64(0xFFFF)
    return (half & np.uint64(127)).astype(np.float64), ((half >> np.uint64(7)) & np.uint64(127)).astype(np.float64)


# -------------------------------------------------------------------- step
def grad(x, scale=1.0, acc=None, coef=1.0):
    """g = (acc + scale x) coef and its bound; x, acc: exact inputs as float64."""
    sx = scale * x
    err = EPS * np.abs(sx)
    g = sx
    if acc is not None:
        g = acc + sx
        err = err + EPS * np.abs(g)
    return g * coef, (err + EPS * np.abs(g)) * abs(coef)


def step(p, m, v, g, g_err, *, lr, b1, b2, eps, wd, t, root=1, div=1):
    """One AdamW step: {name: (value, bound)} for p, m and r = sqrt(v).  root, div: the errors of the
    square root and of the division in EPS (1: correctly rounded; the 8-bit update's Newton root
    and hardware reciprocal: 2 and, with its product, 3)."""
    alpha, bc2 = lr / (1 - b1 ** t), math.sqrt(1 - b2 ** t)
    m1 = b1 * m + (1 - b1) * g
    m_err = EPS * (2 * np.abs(b1 * m) + np.abs((1 - b1) * g) + np.abs(m1)) + (1 - b1) * g_err
    v1 = b2 * v + (1 - b2) * g * g
    # beta2: constant and product; the decoded v is the square of the root, exact in the update; 1 - beta2: constant, product
    v_err = EPS * (2 * b2 * v + 2 * (1 - b2) * g * g + v1) + (1 - b2) * 2 * np.abs(g) * g_err
    r1 = np.sqrt(v1)
    with np.errstate(divide="ignore", invalid="ignore"):
        r_err = np.where(v1 > 0, v_err / (2 * np.maximum(r1, 1e-300)), 0.0)
    d = r1 / bc2 + eps
    # sqrt(1 - beta2^t): constant and division, or its reciprocal's two roundings
    d_err = (r_err + root * EPS * r1) / bc2 + EPS * (2 * r1 / bc2 + eps + d)
    u = m1 / d
    u_err = m_err / d + np.abs(u) * (d_err / d + div * EPS)
    p1 = p * (1 - lr * wd) - alpha * u
    p_err = EPS * (2 * np.abs(p) + 2 * np.abs(alpha * u) + np.abs(p1)) + alpha * u_err
    return {"p": (p1, 1.1 * p_err + TINY), "m": (m1, 1.1 * m_err + TINY), "r": (r1, 1.1 * (r_err + root * EPS * r1) + TINY),
            "v": (v1, 1.1 * v_err + TINY)}


def check_codes(codes, scales, value, bound, *, k=None, floor=False, name=""):
    """The stored codes and scales are what `value`, known to +- bound, rounds to."""
    n = len(codes)
    amax = np.abs(rows(value))
    err = rows(bound)
    lo, hi = scale_of(np.maximum(amax - err, 0).max(1)), scale_of((amax + err).max(1))
    s = scales.astype(np.float64)
    assert np.array_equal(s, np.exp2(np.round(np.log2(s)))), f"{name}: a scale is no power of two"
    assert ((lo <= s) & (s <= hi)).all(), f"{name}: scales"
    per = np.repeat(s, BLOCK)[:n]

    def rounded(x):
        y = x / per
        if floor:
            y = np.where(y > 0, np.maximum(y, 2.0 ** -9), 0.0)
        return grid(y, k)

    got = TABLE[codes]
    a, b = rounded(value - bound), rounded(value + bound)
    if floor:  # the root is known to be >= 0; zero only where the value is
        a = np.where(value > 0, np.maximum(a, 2.0 ** -9), a)
    if k is not None:  # stochastic rounding acts on the size: monotone on each side of zero
        a, b = np.minimum(a, b), np.maximum(a, b)
        near = np.abs(value) <= bound
        a, b = np.where(near, -np.maximum(-a, b), a), np.where(near, np.maximum(-a, b), b)
    bad = ~((a <= got) & (got <= b))
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {n} codes", value[bad][:3], bound[bad][:3], got[bad][:3],
                           (per * got)[bad][:3])


def check_close(got, value, bound, name=""):
    err = np.abs(np.asarray(got, np.float64) - value)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {len(value)}", np.flatnonzero(bad)[:3], err[bad][:3],
                           bound[bad][:3])
