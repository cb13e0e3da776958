"""Caches over which attention is exact, whatever the order of its sums.

Keys and values are the nibbles themselves (s = 1, b = -16). A shown token's key
is zero and a hidden one's at least 8 in some channel; with all queries -1 and
the factor SCALE a shown token's score is 0, so its weight is one power of two,
and a hidden one's at most -8 SCALE log2(e) = -369 in units of log 2, whose
weight beside a shown token is zero in binary32. The sums then are whole numbers
of shown tokens times a power of two, exact in binary32 up to 2^24 of them, and
the output is the mean of the shown tokens' values. Every sequence's first token
is shown, so a row that sees any token sees a shown one.
"""
import numpy as np

from oracle import kv as okv

SCALE = 32.0
ROUND = 2.0 ** -24  # binary32


def tokens(r, shape, D, top=15):
    """Nibbles of random tokens: (kn, vn uint8 (*shape, D), shown bool shape); values up to `top`."""
    shown = r.random(shape) < 0.5
    kn = r.integers(0, 16, (*shape, D), dtype=np.uint8)
    np.put_along_axis(kn, r.integers(0, D, (*shape, 1)), np.uint8(8) + r.integers(0, 8, (*shape, 1), dtype=np.uint8), -1)
    kn[shown] = 0
    return kn, r.integers(0, top + 1, (*shape, D), dtype=np.uint8), shown


def pairs(shape):
    return np.ones((*shape, 1), dtype=np.float16), np.full((*shape, 1), -16, dtype=np.float16)


def pack(kn, vn, page):
    s, b = pairs(kn.shape[:-1])
    return okv.pack(kn, s, b, vn, s, b, page)


def close(got, lse, O, count, f32, sums=2 * ROUND):
    """Whether the outputs (n, D) and log-sum-exps (n,) of rows are the means O of `count` shown tokens (0: none),
    whose sums are known to the relative error `sums` beside the quotient's and the product's rounding."""
    some = count > 0
    bound = np.abs(O) * (sums + 2 * ROUND)
    if not f32:
        bound = bound + np.maximum(np.abs(O) * 2.0 ** -11, 2.0 ** -25)
    ok = (np.abs(got - O) <= bound).all(-1) & (some | (got == 0).all(-1))
    # lse = (-12 + log2(2^12 count)) ln 2: the logarithm, below 64, to a unit in its last place (2^-18), a product of
    # a rounded constant
    want = np.where(some, np.log(np.maximum(count, 1)), okv.LOWEST)
    return ok & np.where(some, np.abs(lse - want) <= 2.0 ** -18 + sums + np.abs(want) * 2 * ROUND, lse == okv.LOWEST)


class Sequences:
    """A cache of sequences of these lengths, pages shuffled, the bytes of no sequence NaN pairs; what their rows are."""

    def __init__(self, seed, Hkv, D, page, lens, top=15):
        r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        ids = r.permutation(sum(need) + 1).astype(np.int32)
        slots = (sum(need) + 1) * page
        kn, vn, shown = tokens(r, (slots, Hkv), D, top)
        self.table = np.full((len(lens), max(1, max(need))), -7, dtype=np.int32)  # nothing reads the rest
        self.shown, self.values, used, at = [], [], np.zeros(slots, dtype=bool), 0
        for i, n in enumerate(lens):
            self.table[i, :need[i]] = ids[at:at + need[i]]
            at += need[i]
            slot = (self.table[i, :need[i], None].astype(np.int64) * page + np.arange(page)).reshape(-1)[:n]
            kn[slot[:1]], shown[slot[:1]], used[slot] = 0, True, True
            self.shown.append(shown[slot])
            self.values.append(vn[slot])
        s, b = pairs((slots, Hkv))
        s[~used], b[~used] = np.nan, np.nan
        self.pages = okv.pack(kn, s, b, vn, s, b, page)

    def rows(self, i, seen, G):
        """(O (n, Hq, D), count (n, Hq)) of rows of sequence i that see the first seen[n] tokens."""
        shown, values = self.shown[i], self.values[i]
        if len(shown) == 0:
            shown, values = np.zeros((1, *shown.shape[1:]), dtype=bool), np.zeros((1, *values.shape[1:]), dtype=np.uint8)
        last = np.maximum(np.asarray(seen) - 1, 0)
        least, span = last.min(initial=0), last.max(initial=0) + 1
        kept = values * shown[..., None]
        count, total = shown[:least].sum(0, dtype=np.int64), kept[:least].sum(0, dtype=np.int64)
        count = count + np.cumsum(shown[least:span], 0, dtype=np.int64)[last - least]
        total = total + np.cumsum(kept[least:span], 0, dtype=np.int64)[last - least]
        count[np.asarray(seen) <= 0] = 0
        O = np.where(count[..., None] > 0, total / np.maximum(count, 1)[..., None], 0.0)
        return np.repeat(O, G, 1), np.repeat(count, G, 1)
