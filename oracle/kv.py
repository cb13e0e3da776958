"""CPU oracle for the 4-bit paged key/value cache (test infrastructure only).

Plain numpy in binary64 from the definitions in include/kvcache.h; it shares
nothing with the GPU path. ``pack`` and ``unpack`` walk the page layout nibble
by nibble as the header words it.
"""
from __future__ import annotations

import numpy as np

LOWEST = float(np.finfo(np.float32).min)  # log-sum-exp of a row that sees no token
LIMIT = 20000.0


def norm(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def rope(x, table_rows, interleaved):
    """x (T, H, D) rotated by table_rows (T, R): R / 2 cosines, then R / 2 sines."""
    x = np.array(x, dtype=np.float64)
    R = table_rows.shape[1]
    cos, sin = (np.asarray(t, dtype=np.float64)[:, None] for t in (table_rows[:, :R // 2], table_rows[:, R // 2:]))
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    u, y = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * cos - y * sin
    x[..., b] = y * cos + u * sin
    return x


def quantise(x):
    """(n uint8, s float16, b float16, t): the 4-bit form of the last axis of x; t is (x - b) / s - 16 before
    it is rounded and clamped."""
    x = np.clip(np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=LIMIT, neginf=-LIMIT), -LIMIT, LIMIT)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    s = ((hi - lo) / 15).astype(np.float32).astype(np.float16)
    sd = s.astype(np.float64)
    b = (lo - 16 * sd).astype(np.float32).astype(np.float16)
    t = np.where(sd > 0, (x - b.astype(np.float64)) / np.where(sd > 0, sd, 1), 16) - 16
    return np.clip(np.rint(t), 0, 15).astype(np.uint8), s, b, t


def held(n, s, b):
    """The binary16 values that nibbles stand for, as binary64 (16 + n and s have 5 and 11 bits: the sum is exact
    in binary64 unless it is out of binary16's reach anyway, so it is rounded once)."""
    return ((16.0 + n) * s.astype(np.float64) + b.astype(np.float64)).astype(np.float16).astype(np.float64)


def _places(D):
    """Byte and shift in a block of token t's channel d, for keys and values, and bytes of their (s, b)."""
    t, d = np.arange(32)[:, None], np.arange(D)[None, :]
    kbyte, kshift = t * (D // 2) + d // 2 + 0 * t, 4 * (d % 2) + 0 * t
    h, q, i = t // 16, t // 4 % 4, t % 4
    c, g, j = d // (D // 16), d % (D // 16) // 4, d % 4
    word = ((g * 4 + q) * 16 + c) * 8 + 4 * h + i
    vbyte, vshift = 16 * D + 2 * word + j // 2, 4 * (j % 2) + 0 * t
    t = t[:, 0]
    pairs = 32 * D
    at = pairs + 128 + 2 * (8 * (t // 4 % 4) + 4 * (t // 16) + t % 4)
    return (kbyte, kshift), (vbyte, vshift), (pairs + 4 * t, pairs + 4 * t + 2), (at, at + 64)


def unpack(pages, Hkv, D, page_tokens):
    """Nibbles and pairs of every slot: kn, vn (slots, Hkv, D) uint8, ks, kb, vs, vb (slots, Hkv, 1) float16."""
    pages = np.ascontiguousarray(pages, dtype=np.uint8)
    P, nb, size = pages.shape[0], page_tokens // 32, 32 * (D + 8)
    blk = pages.reshape(P, Hkv, nb, size)
    k, v, kp, vp = _places(D)
    out = []
    for byte, shift in (k, v):
        out.append((blk[..., byte] >> shift.astype(np.uint8)) & 15)  # (P, Hkv, nb, 32, D)
    par = []
    for at in (*kp, *vp):
        raw = np.stack([blk[..., at], blk[..., at + 1]], -1).copy()
        par.append(raw.view(np.float16))  # (P, Hkv, nb, 32, 1)
    order = lambda x: x.transpose(0, 2, 3, 1, 4).reshape(P * page_tokens, Hkv, x.shape[-1])  # noqa: E731
    kn, vn = (order(x) for x in out)
    ks, kb, vs, vb = (order(x) for x in par)
    return kn, ks, kb, vn, vs, vb


def pack(kn, ks, kb, vn, vs, vb, page_tokens):
    """Pages (P, page_bytes) uint8 of the nibbles and pairs of P * page_tokens slots (inverse of unpack)."""
    S, Hkv, D = kn.shape
    P, nb, size = S // page_tokens, page_tokens // 32, 32 * (D + 8)
    blk = np.zeros((P, Hkv, nb, size), dtype=np.uint8)
    place = lambda x: x.reshape(P, nb, 32, Hkv, x.shape[-1]).transpose(0, 3, 1, 2, 4)  # noqa: E731
    k, v, kp, vp = _places(D)
    for (byte, shift), n in ((k, kn), (v, vn)):
        n = place(n)
        for t in range(32):
            for s in (0, 4):  # no two channels share a half
                here = shift[t] == s
                blk[..., byte[t][here]] |= (n[..., t, :][..., here] << np.uint8(s)).astype(np.uint8)
    for at, x in zip((*kp, *vp), (ks, kb, vs, vb)):
        raw = np.ascontiguousarray(place(x)).view(np.uint8)
        blk[..., at], blk[..., at + 1] = raw[..., 0], raw[..., 1]
    return blk.reshape(P, Hkv * nb * size)


def attend(q, K, V, seen, scale):
    """Attention of one sequence. q (n, Hq, D); K, V (L, Hkv, D); seen (n,): row i sees the first seen[i] tokens.
    Returns (O (n, Hq, D), lse (n, Hq), mass (n, Hq, D), reach (n, Hq)) in binary64: mass = sum p |v| / sum p and
    reach = the largest sum_d |scale q_d k_d|, which rounding bounds are made of."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    n, Hq, D = q.shape
    G = Hq // K.shape[1]
    O, lse = np.zeros((n, Hq, D)), np.full((n, Hq), LOWEST)
    mass, reach = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        L = int(seen[i])
        if L <= 0:
            continue
        for h in range(Hq):
            k, v = K[:L, h // G], V[:L, h // G]
            s = scale * (k @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            O[i, h] = p @ v / p.sum()
            mass[i, h] = p @ np.abs(v) / p.sum()
            lse[i, h] = m + np.log(p.sum())
            reach[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return O, lse, mass, reach
