"""The verification oracle against exact fractions, and these against the target's distribution (no GPU).

tests/kv_fractions.py follows the definition in rational numbers, where the distribution of what comes out can be
compared without a tolerance; the oracle's borders, found by bisection of its random numbers, are compared with its.
"""
import inspect
from fractions import Fraction

import numpy as np
import pytest

from oracle import kvtree as okt
from tests import kv_fractions as kf

STEP = 2.0 ** -24
P = [16 / 32, 2 / 32, 5 / 32, 9 / 32]
Q = [3 / 32, 19 / 32, 8 / 32, 2 / 32]
# A draft sure of its first token, as binary32 holds it: the row's sum is off 1 by a third of what is left of it.
SURE_P, SURE_Q = [0.3, 0.5, 0.2], [1 - 2 * STEP, 2 * STEP, STEP]


def border(below, top=1.0):
    """The largest number below which below() holds, by bisection: to 2^-52."""
    lo, hi = 0.0, top
    for _ in range(54):
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if below(mid) else (lo, mid)
    return hi


def borders(verify, p, q, drafts):
    """star's numbers, of a verification."""
    kids = len(drafts)
    rows = [np.repeat(np.array([x]), kids + 1, 0) if x is not None else None for x in (p, q)]
    tree = (0,) + tuple(drafts), [-1] + [0] * kids, *rows
    u, out = [0.0] + [okt.BELOW_ONE] * kids, []
    for c in range(1, kids + 1):
        def taken(x):
            return verify(*tree, u[:c] + [x] + u[c + 1:])[0] == [0, c]
        if taken(okt.BELOW_ONE):
            return out + [1.0], None
        out.append(border(taken, okt.BELOW_ONE))
    sums = [border(lambda x: verify(*tree, [x] + u[1:])[1] <= t) for t in range(len(p) - 1)] + [1.0]
    return out, np.diff([0.0] + sums)


def off(verify, p, q, drafts):
    """The farthest that a border lies from the exact one."""
    want, weights = kf.star(p, q, drafts)
    got, drawn = borders(verify, p, q, drafts)
    if len(got) != len(want) or (drawn is None) != (want[-1] == 1):
        return 1.0
    far = max(abs(a - float(b)) for a, b in zip(got, want))
    if drawn is not None:
        far = max(far, max(abs(a - float(b / sum(weights))) for a, b in zip(drawn, weights)))
    return far


@pytest.mark.parametrize("kids", [1, 2, 3])
@pytest.mark.parametrize("drawn", [True, False])
def test_fractions_give_the_targets_distribution(drawn, kids):
    got = [Fraction(0)] * 4
    for drafts, chance in kf.orders(Q, kids):
        one = kf.first_token(*kf.star(P, Q if drawn else None, drafts), drafts)
        if not drawn:
            assert one == kf.fractions(P)
        got = [a + chance * b for a, b in zip(got, one)]
    assert got == kf.fractions(P)


def test_fractions_of_a_sure_draft_give_the_targets_distribution():
    """Its row counts as a sum of 1, from which it is STEP away: so may the distribution be."""
    got = [0.0] * 3
    for drafts, chance in kf.orders(SURE_Q, 2):
        got = [a + float(chance * b) for a, b in zip(got, kf.first_token(*kf.star(SURE_P, SURE_Q, drafts), drafts))]
    np.testing.assert_allclose(got, SURE_P, atol=2 * STEP)


def cases():
    for kids in (1, 2, 3):
        for drafts, _ in kf.orders(Q, kids):
            yield P, Q, drafts
            yield P, None, drafts
    for drafts, _ in kf.orders(SURE_Q, 2):
        yield SURE_P, SURE_Q, drafts


def test_the_oracles_borders_are_the_exact_ones():
    # borders are ratios of up to ten rounded numbers and sums, no less than a 16th of their terms; the bisection's 2^-52
    for p, q, drafts in cases():
        assert off(okt.verify, p, q, drafts) < 1e-13, (q is None, drafts)


@pytest.mark.parametrize("right,wrong,drawn", [
    ("draft = d / mass", "draft = d", True),                               # the draft's rest is not normalised
    ("mass = d.sum()", "mass = 1.0 - unit(q[cur])[tried[0]]", True),      # by the first rejected token only
    ("mass = d.sum()", "mass = 1.0 - sum(unit(q[cur])[t] for t in tried)", True),  # as if the row's sum were 1
    ("left = w.sum()", "pass", True),                                     # the target's rest is not normalised
    ("left -= w[x]", "pass", False),
    ("d[x] = 0.0", "pass", True),                                         # the draft keeps a rejected token
    ("w[x] = 0.0", "pass", False),
])
def test_mistakes_show(right, wrong, drawn):
    source = inspect.getsource(okt.verify)
    assert source.count(right) == 1
    scope = dict(vars(okt))
    exec(source.replace(right, wrong), scope)
    assert max(off(scope["verify"], p, q, drafts) for p, q, drafts in cases() if (q is not None) == drawn) > 1e-2
