"""Verification of one node's drafts (include/kvcache.h, kvc_verify) in exact fractions, from the definition itself."""
from __future__ import annotations

import itertools
from fractions import Fraction


def fractions(x):
    return [Fraction(float(v)) for v in x]


def star(p, q, drafts):
    """(thresholds, weights): child j is accepted if u[j] < thresholds[j], given that those before it were not; then the
    weights that the last token is drawn from. q None: the drafts are certain. A whole row counts as a sum of 1."""
    w, left = fractions(p), Fraction(1)
    d, mass = None if q is None else fractions(q), Fraction(1)
    out = []
    for x in drafts:
        draft = [Fraction(t == x) for t in range(len(w))] if q is None else [v / mass for v in d]
        out.append(min(Fraction(1), w[x] / (left * draft[x])))
        before = w[x]
        w = [max(Fraction(0), a - left * b) for a, b in zip(w, draft)]
        if q is None:
            left -= before
        else:
            left = sum(w)
            d[x] = Fraction(0)
            mass = sum(d)
        if out[-1] == 1:
            break
    return out, w


def orders(q, kids):
    """Every order of `kids` tokens that a draft can draw without replacement, and its chance."""
    q = fractions(q)
    for drafts in itertools.permutations([t for t, v in enumerate(q) if v], kids):
        chance, left = Fraction(1), sum(q)
        for x in drafts:
            chance *= q[x] / left
            left -= q[x]
        yield drafts, chance


def first_token(thresholds, weights, drafts):
    """The distribution of the first token that comes out, for these drafts."""
    out, reach = [Fraction(0)] * len(weights), Fraction(1)
    for t, x in zip(thresholds, drafts):
        out[x] += reach * t
        reach *= 1 - t
    if reach:
        total = sum(weights)
        out = [a + reach * b / total for a, b in zip(out, weights)]
    return out
