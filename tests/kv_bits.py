"""Rows that decide how the 4-bit form is rounded, and what their nibbles and pairs have to be, bit for bit."""
import numpy as np

from oracle import kv as okv


def _f16(x):
    return x.astype(np.float32).astype(np.float16)


def rows(seed, n, D):
    """About n binary16 rows of D: ordinary ones, and ones whose numbers lie on the borders between two roundings."""
    r = np.random.default_rng(seed)
    m = n // 6
    out = [(r.standard_normal((n - 5 * m, D)) * np.exp2(r.integers(-9, 10, (n - 5 * m, 1)))).astype(np.float16)]
    # (x - b) / s a whole number and a half, everywhere: s = 2 u, the row from o - 15 u to o + 15 u in steps of u, an
    # odd number (1 / s is not one of binary32) times a power of two
    u = (2 * r.integers(0, 17, (m, 1)) + 1) * np.exp2(r.integers(-13, -1, (m, 1)))
    x = r.integers(0, 31, (m, D))
    x[:, 0], x[:, 1] = 0, 30
    out.append(((x - 15 + 2 * r.integers(-14, 15, (m, 1))) * u).astype(np.float16))
    # (max - min) / 15 = 1 + (2 k + 1) / 2^11, half way between two binary16 numbers, and next to that
    k = r.integers(0, 68, (m, 1))
    lo = (-15.0 * (2 * k + 1) / 2048).astype(np.float16)
    bits = (lo.view(np.uint16) + r.integers(-1, 2, (m, 1)).astype(np.int16).view(np.uint16)).astype(np.uint16)
    x = r.uniform(0, 15, (m, D)).astype(np.float16)
    x[:, :1], x[:, 1:2] = bits.view(np.float16), 15
    out.append(x)
    # s = 1 and min x - 16 half way between two binary16 numbers of 8 .. 16
    lo = (2 * r.integers(0, 1000, (m, 1)) + 1) / 256
    x = r.uniform(lo, lo + 14.9, (m, D)).astype(np.float16)
    x[:, :1], x[:, 1:2] = lo, lo + 15
    out.append(x)
    # few bits: ties of all kinds
    out.append((r.integers(-24, 25, (m, D)) * np.exp2(r.integers(-24, 9, (m, 1)))).astype(np.float16))
    # a large number beside small ones, constants and zeros
    x = r.standard_normal((m, D)) * 2.0 ** -8
    x[:, 0] = r.choice([20000, -20000, 1000, -3, 0.5, 0], m)
    x[::7] = x[::7, :1]
    x[3::7] = 0
    out.append(x.astype(np.float16))
    for y in out:  # the extremes anywhere in the row
        r.permuted(y, axis=-1, out=y)
    return np.concatenate(out)


def exact(x, n, s, b):
    """Whether (n, s, b) is the 4-bit form of rows of binary16 numbers x, for each row."""
    on, os_, ob, _ = okv.quantise(x)
    return ((n == on).all(-1) & (s.view(np.uint16) == os_.view(np.uint16))[..., 0] &
            (b.view(np.uint16) == ob.view(np.uint16))[..., 0])


def near(x, n, s, b, off=1e-12):
    """The same for rows x of binary64 numbers known to `off` times the row's largest: a pair or a nibble may be either
    of two only where x, that far off, gives either."""
    d = off * np.abs(x).max(-1, keepdims=True)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    between = lambda v, least, most: (least <= v) & (v <= most)  # noqa: E731
    ok = between(s, _f16((hi - lo - 2 * d) / 15), _f16((hi - lo + 2 * d) / 15))
    sd = s.astype(np.float64)
    ok &= between(b, _f16(lo - 16 * sd - d), _f16(lo - 16 * sd + d))
    step = np.where(sd > 0, sd, 1)
    t = lambda e: np.clip(np.rint(np.where(sd > 0, (x + e - b.astype(np.float64)) / step - 16, 0)), 0, 15)  # noqa: E731
    return ok[..., 0] & between(n, t(-d), t(d)).all(-1)
