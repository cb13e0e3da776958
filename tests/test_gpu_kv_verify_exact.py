"""GPU verification of siblings at the exact borders of their decisions (tests/kv_fractions.py)."""
import numpy as np
import pytest

from tests import kv_fractions as kf
from tests import test_kv_verify_exact as exact
from tests.test_gpu_kv import _cache
from tests.test_gpu_kv_tree import _run_verify, _starts

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -20  # the binary32 random numbers and rows are off by 2^-25 at most, the sums by less
ALMOST = float(np.float32(1) - np.float32(2.0 ** -24))


def _decisions(thresholds, weights):
    """Random numbers of node 0 and the children, and what comes of them: (u, accepted child or 0, token or None)."""
    kids = len(thresholds)
    for c, t in enumerate(thresholds):
        for u, taken in ((float(t) - NEAR, True), (float(t) + NEAR, False)):
            if 0 <= u < ALMOST and (taken or c + 1 == kids):
                yield [0.5] + [ALMOST] * c + [u] + [0.0 if taken else ALMOST] * (kids - c - 1), c + 1 if taken else 0, None
    if thresholds[-1] < 1 - 2 * NEAR:
        total, at = sum(weights), 0
        for token, w in enumerate(weights):
            if w / total > 3 * NEAR:
                for u in (float(at / total) + NEAR, float((at + w) / total) - NEAR):
                    yield [u] + [ALMOST] * kids, 0, token
            at += w


def _problem(cases, tokens, vocab):
    """All decisions of all cases (p, q, drafts) as one batch; their tokens are `tokens` of the vocabulary."""
    drafts, us, want, rows = [], [], [], []
    for p, q, order in cases:
        p, q = (None if x is None else np.asarray(x, dtype=np.float32) for x in (p, q))
        thresholds, weights = kf.star(p, q, order)
        for u, child, token in _decisions(thresholds, weights):
            # a child behind one that is always accepted is never tried
            drafts.append([0] + [tokens[x] for x in order])
            us.append(u + [0.5] * (len(order) + 1 - len(u)))
            want.append((child, None if token is None else tokens[token]))
            rows.append((p, q))
    sizes = [len(d) for d in drafts]
    T = sum(sizes)
    starts = _starts(sizes)
    p, q = np.zeros((T, vocab), dtype=np.float32), np.zeros((T, vocab), dtype=np.float32)
    for b, (a, d) in enumerate(rows):
        p[starts[b]:starts[b + 1], tokens] = a
        if d is not None:
            q[starts[b]:starts[b + 1], tokens] = d
    return dict(T=T, starts=starts, token=np.concatenate(drafts), parent=np.concatenate([[-1] + [0] * (n - 1) for n in sizes]),
                p=p, q=None if rows[0][1] is None else q, u=np.concatenate(us).astype(np.float32)), want


def _check(got, c, want):
    path, count, nxt = got
    for b, (child, token) in enumerate(want):
        assert path[c["starts"][b]:c["starts"][b + 1]].tolist()[:2][1:] == ([child] if child else [-1]), b
        assert count[b] == 1 + (child > 0)
        assert token is None or nxt[b] == token, (b, nxt[b], token)


@pytest.mark.parametrize("children", [1, 3])
@pytest.mark.parametrize("tokens,vocab", [([0, 1, 2, 3], 4), ([5, 2047, 2048, 9000], 9001)])
@pytest.mark.parametrize("drawn", [True, False])
def test_siblings_are_held_against_the_exact_borders(drawn, tokens, vocab, children):
    print(f"[kv verify exact] {drawn} {vocab} {children}", flush=True)
    kv = _cache(1, 1, 64)
    four = [x for x in exact.cases() if len(x[0]) == 4 and (x[1] is not None) == drawn]
    three = [x for x in exact.cases() if len(x[0]) == 3] if drawn else []
    for cases, at in ((four, tokens), (three, tokens[:3])):
        if cases:
            c, want = _problem(cases, at, vocab)
            got = _run_verify(kv, c, max_children=children)
            kv.check()
            _check(got, c, want)


@pytest.mark.parametrize("children", [1, 3])
@pytest.mark.parametrize("left", [1e-4, 1e-9, 2e-12, 1e-15])
def test_siblings_of_a_draft_that_leaves_next_to_nothing(left, children):
    """The draft's first token has all of binary32's 1, the others share `left`, much of it in entries below 2^-51; the
    second draft is held against its part of that, or passed over where nothing counts as left."""
    print(f"[kv verify rest] {left} {children}", flush=True)
    kv = _cache(1, 1, 64)
    V, r = 6000, np.random.default_rng(8)
    q = r.random(V) ** 4
    q = (q * (left / q.sum())).astype(np.float32)
    q[4000] = 1.0
    p = r.random(V) ** 4
    p = (p * (0.7 / (p.sum() - p[4000]))).astype(np.float32)
    p[4000] = 0.3
    gone = left < V * 2.0 ** -57
    drafts = []
    for x in r.permutation(V):
        if x != 4000 and q[x]:
            if 0.05 < float(p[x]) / 0.7 / (float(q[x]) / left) < 0.95:
                drafts.append((4000, int(x)))
        if len(drafts) == 3:
            break
    cases = []
    for order in drafts:
        thresholds, weights = kf.star(p, q, order)
        assert 0.04 < thresholds[1] < 0.96
        if gone:
            for u in (0.0, float(thresholds[1]) - NEAR):
                cases.append(([0.5, ALMOST, u], order, 0))
        else:
            for u, child in ((float(thresholds[1]) - NEAR, 2), (float(thresholds[1]) + NEAR, 0)):
                cases.append(([0.5, ALMOST, u], order, child))
    n = len(cases)
    c = dict(T=3 * n, starts=_starts([3] * n), token=np.concatenate([[0, *order] for _, order, _ in cases]),
             parent=[-1, 0, 0] * n, p=np.repeat(p[None], 3 * n, 0), q=np.repeat(q[None], 3 * n, 0),
             u=np.concatenate([u for u, _, _ in cases]).astype(np.float32))
    got = _run_verify(kv, c, max_children=children)
    kv.check()
    _check(got, c, [(child, None) for _, _, child in cases])
