"""CPU oracle for a step with drafted tokens on the key/value cache (test infrastructure only).

Plain Python and numpy in binary64 from the definitions in include/kvcache.h; it
shares nothing with the GPU path.
"""
from __future__ import annotations

import numpy as np

from oracle.kv import LOWEST

BELOW_ONE = float(np.float32(1) - np.float32(2.0 ** -24))


def ancestors(parent):
    """For each node, itself and its ancestors."""
    out = []
    for i, p in enumerate(parent):
        out.append({i} | (out[p] if 0 <= p < i else set()))
    return out


def masks(parent, words):
    """(n, words) uint64."""
    out = np.zeros((len(parent), words), dtype=np.uint64)
    for i, nodes in enumerate(ancestors(parent)):
        for j in nodes:
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out


def visible(mask, off, length):
    """(n, length) bool: token t of a sequence is seen by the row with this mask."""
    t = np.arange(length)
    node = t - off
    inside = (node >= 0) & (node < 64 * mask.shape[1])
    at = np.where(inside, node, 0)
    bit = (mask[:, at // 64] >> (at % 64).astype(np.uint64)) & np.uint64(1)
    return (node < 0)[None] | (inside[None] & (bit == 1))


def attend(q, K, V, seen, scale):
    """Attention of one sequence. q (n, Hq, D); K, V (L, Hkv, D); seen (n, L) bool. Returns (O, lse, mass, reach) as
    oracle.kv.attend does."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    n, Hq, D = q.shape
    G = Hq // K.shape[1]
    O, mass = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, reach = np.full((n, Hq), LOWEST), np.zeros((n, Hq))
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        s = np.where(seen, scale * (q[:, h] @ k.T), -np.inf)
        for i in range(n):
            if not seen[i].any():
                continue
            m = s[i].max()
            p = np.exp(s[i] - m)
            O[i, h], mass[i, h] = p @ v / p.sum(), p @ np.abs(v) / p.sum()
            lse[i, h] = m + np.log(p.sum())
            reach[i, h] = abs(scale) * (np.abs(k[seen[i]]) @ np.abs(q[i, h])).max()
    return O, lse, mass, reach


def unit(x):
    return np.clip(np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0), 0.0, 1.0)


def verify(token, parent, p, q, u):
    """(path, next, margin) of one tree, by the distributions themselves, child by child. next is -1 where p has no
    weight. margin: how near the closest decision was, relative to what was compared."""
    n, vocab = len(parent), p.shape[1]
    u = [min(max(float(x), 0.0), BELOW_ONE) if x == x else 0.0 for x in u]
    path, margin = [0], 1.0
    while True:
        cur, taken, tried = path[-1], None, []
        w, left = unit(p[cur]), 1.0             # the target's weights, and their sum (a whole row counts as 1)
        d = None if q is None else unit(q[cur])  # the draft's, without the tried tokens
        for c in range(cur + 1, n):
            x = int(token[c])
            if parent[c] != cur or not 0 <= x < vocab or x in tried or not left > 0:
                continue
            if q is None:
                draft = np.zeros(vocab)
                draft[x] = 1.0
            else:
                mass = 1.0  # a whole row counts as 1
                if tried:
                    mass = d.sum()
                if not mass > vocab * 2.0 ** -57:
                    continue
                draft = d / mass
            tried.append(x)
            a, b = u[c] * draft[x], w[x] / left
            margin = min(margin, abs(a - b) / max(a, b, 1e-300))
            if a < b:
                taken = c
                break
            if q is None:  # all of x, which leaves the others in proportion
                left -= w[x]
                w[x] = 0.0
            else:
                w = np.maximum(0.0, w - left * draft)
                left = w.sum()
                d[x] = 0.0
        if taken is None:
            break
        path.append(taken)
    if not w.sum() > 0:
        w = unit(p[cur])
    sums = np.cumsum(w)
    if not sums[-1] > 0:
        return path, -1, margin
    at = u[0] * sums[-1]
    nxt = int(np.searchsorted(sums, at, side="right"))
    near = min(sums[nxt] - at, at - sums[nxt - 1] if nxt else 1.0)
    return path, nxt, min(margin, near / sums[-1])
