"""GPU tests of the 4-bit paged key/value cache (include/kvcache.h) against the binary64 oracle.

Tolerances count roundings: a rounding to binary16 is off by at most 2^-11 of
the value (2^-25 where it is subnormal), to binary32 by 2^-24.
"""
import numpy as np
import pytest

from oracle import fd as fdo
from oracle import kv as okv
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _half(y):
    """Half a step of binary16 at y."""
    return np.maximum(np.abs(y) * 2.0 ** -11, 2.0 ** -25)


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(gu.dev())


def _cache(*shape, **kw):
    from shard_decomposed_gemm_amd import KvCache
    return KvCache(*shape, **kw)


# ---------------------------------------------------------------- append

def _table(length, R):
    """Cosines and sines of position * 10000^(-2 i / R) in binary32."""
    a = np.arange(length)[:, None] * 10000.0 ** (-2 * np.arange(R // 2) / R)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _append_case(seed, T, Hq, Hkv, D, R, interleaved, norm, length=5000, scale=1.0):
    r = np.random.default_rng(seed)
    x = (scale * r.standard_normal((T, Hq + 2 * Hkv, D)) * np.exp(0.7 * r.standard_normal((1, Hq + 2 * Hkv, D))))
    c = dict(x=x.astype(np.float16), pos=r.integers(0, length, T), table=_table(length, R) if R else None, R=R,
             interleaved=interleaved, qw=None, kw=None)
    if norm:
        c["qw"], c["kw"] = ((1 + 0.3 * r.standard_normal(D)).astype(np.float16) for _ in range(2))
    return c


def _append_expected(c, Hq, Hkv, eps=1e-6):
    """(q_out, K, V) in binary64 and a bound on the binary32 error of q and K before they are rounded."""
    x = c["x"].astype(np.float64)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if c["qw"] is not None:
        q, k = okv.norm(q, c["qw"], eps), okv.norm(k, c["kw"], eps)
    # norm: a sum of D squares over 16 lanes (D / 16 + 4 additions), a root, a quotient, three products;
    # rotation: two products and a sum on values of the row's largest size
    err = lambda y: np.abs(y).max(-1, keepdims=True) * (y.shape[-1] / 16 + 16) * 2.0 ** -23  # noqa: E731
    eq, ek = err(q), err(k)
    if c["R"]:
        rows = c["table"][c["pos"]]
        q, k = okv.rope(q, rows, c["interleaved"]), okv.rope(k, rows, c["interleaved"])
    return q, k, v, eq, ek


def _check_rows(x, err, n, s, b):
    """The stored 4-bit rows (n, s, b) against what binary64 says of x, known to `err`."""
    on, os_, ob, t = okv.quantise(x)
    xc = np.clip(x, -okv.LIMIT, okv.LIMIT)
    sd, bd = s.astype(np.float64), b.astype(np.float64)
    bound = sd / 2 + 15 * _half(sd) + _half(bd) + _half(np.abs(xc) + sd) + 4 * err + 2.0 ** -18 * sd
    assert (np.abs(okv.held(n, s, b) - xc) <= bound).all()
    same = (s == os_) & (b == ob)
    rows = same.size
    assert rows - same.sum() <= 1 + rows // 50, "pairs that differ"
    # equal pairs: a nibble may only differ by one, where x lies next to the border between two
    near = np.abs(t - np.floor(t) - 0.5) <= 2 * err / np.maximum(sd, 1e-30) + 2.0 ** -17
    off = (n != on) & same
    assert (off <= (near & (np.abs(n.astype(int) - on) == 1))).all()
    assert off.sum() <= off.size / 100


APPENDS = [
    # T, Hq, Hkv, D, page, R, interleaved, norm
    (1, 64, 8, 128, 64, 128, False, False),
    (1, 1, 1, 64, 32, 64, False, True),
    (37, 12, 4, 128, 32, 128, False, True),
    (130, 5, 5, 64, 64, 32, True, False),
    (65, 16, 2, 256, 128, 256, False, True),
    (33, 6, 3, 256, 256, 32, True, True),
    (50, 8, 8, 64, 256, 8, False, False),
    (41, 24, 2, 128, 64, 112, False, True),
    (29, 3, 1, 128, 64, 16, True, False),
    (40, 7, 7, 128, 32, 0, False, True),
    (700, 96, 8, 128, 64, 128, True, True),
    (4999, 6, 3, 64, 64, 64, False, False),
    (2050, 16, 2, 128, 128, 64, True, True),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,page,R,interleaved,norm", APPENDS)
def test_append_against_the_oracle(T, Hq, Hkv, D, page, R, interleaved, norm):
    import torch
    print(f"[kv append] {T} {Hq} {Hkv} {D} {page} {R} {interleaved} {norm}", flush=True)
    c = _append_case(T + D, T, Hq, Hkv, D, R, interleaved, norm)
    r = np.random.default_rng(T)
    P = -(-T // page) + 2
    slots = r.permutation(P * page)[:T].astype(np.int64)
    slots[r.random(T) < 0.1] = -1
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=P)
    before = r.integers(0, 256, (P, kv.page_bytes), dtype=np.uint8)
    pages, x = _dev(before), _dev(c["x"])
    q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.float16, device=gu.dev())
    opt = {k: _dev(v) for k, v in (("q_norm", c["qw"]), ("k_norm", c["kw"]), ("rope", c["table"])) if v is not None}
    kv.append(pages, q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], slots=_dev(slots), positions=_dev(c["pos"]),
              interleaved=interleaved, q_out=q_out, **opt)
    k_out, v_out = (torch.full((T, Hkv, D), 7.0, dtype=torch.float16, device=gu.dev()) for _ in range(2))
    kv.read(pages, _dev(slots), k_out, v_out)
    torch.cuda.synchronize()
    kv.check()
    q, k, v, eq, ek = _append_expected(c, Hq, Hkv)
    got = q_out.cpu().numpy().astype(np.float64)
    assert (np.abs(got - q) <= _half(np.abs(q) + eq) + 2 * eq).all()
    kn, ks, kb, vn, vs, vb = okv.unpack(pages.cpu().numpy(), Hkv, D, page)
    keep = slots >= 0
    at = slots[keep]
    _check_rows(k[keep], ek[keep], kn[at], ks[at], kb[at])
    _check_rows(v[keep], 0.0, vn[at], vs[at], vb[at])
    # every other slot is as it was
    was = okv.unpack(before, Hkv, D, page)
    other = np.setdiff1d(np.arange(P * page), at)
    for new, old in zip((kn, ks, kb, vn, vs, vb), was):
        np.testing.assert_array_equal(new[other].view(np.uint8), old[other].view(np.uint8))
    # read gives the values that the stored nibbles stand for, and leaves the rows of negative slots
    np.testing.assert_array_equal(k_out.cpu().numpy()[keep].astype(np.float64), okv.held(kn[at], ks[at], kb[at]))
    np.testing.assert_array_equal(v_out.cpu().numpy()[keep].astype(np.float64), okv.held(vn[at], vs[at], vb[at]))
    assert (k_out.cpu().numpy()[~keep] == 7).all() and (v_out.cpu().numpy()[~keep] == 7).all()


def test_append_parts_in_place_and_broadcast():
    """Queries alone in place, keys and values alone, and one key row broadcast over the tokens."""
    import torch
    T, Hq, Hkv, D = 9, 4, 2, 128
    c = _append_case(3, T, Hq, Hkv, D, 128, False, True)
    q, k, v, eq, ek = _append_expected(c, Hq, Hkv)
    kv = _cache(Hq, Hkv, D, page_tokens=32, num_pages=2)
    x, table, pos = _dev(c["x"]), _dev(c["table"]), _dev(c["pos"])
    kv.append(None, q=x[:, :Hq], q_out=x[:, :Hq], positions=pos, rope=table, q_norm=_dev(c["qw"]))
    torch.cuda.synchronize()
    got = x.cpu().numpy()
    assert (np.abs(got[:, :Hq] - q) <= _half(np.abs(q) + eq) + 2 * eq).all()
    np.testing.assert_array_equal(got[:, Hq:], c["x"][:, Hq:])
    pages = kv.new_pages()
    slots = np.arange(40, 40 + T)
    kv.append(pages, k=x[:1, Hq:Hq + Hkv].expand(T, Hkv, D), v=x[:, Hq + Hkv:], slots=_dev(slots))
    torch.cuda.synchronize()
    kv.check()
    kn, ks, kb, vn, vs, vb = okv.unpack(pages.cpu().numpy(), Hkv, D, 32)
    raw = c["x"].astype(np.float64)
    _check_rows(np.repeat(raw[:1, Hq:Hq + Hkv], T, 0), 0.0, kn[slots], ks[slots], kb[slots])
    _check_rows(v, 0.0, vn[slots], vs[slots], vb[slots])
    kv.append(pages, k=x[:0, Hq:Hq + Hkv], v=x[:0, Hq + Hkv:], slots=_dev(slots[:0]))  # nothing


def test_append_odd_values():
    """Constant rows, zero rows, tiny and huge numbers, infinities and NaN: the cache holds finite numbers."""
    import torch
    D = 128
    x = np.zeros((6, 1, D), dtype=np.float16)
    x[1] = 0.625
    x[2] = (np.arange(D) % 3 - 1) * 2.0 ** -24
    x[3, 0, ::2] = 65504
    x[4, 0, :3] = np.inf, -np.inf, np.nan
    x[5] = np.linspace(-19000, 19000, D)
    kv = _cache(1, 1, D, page_tokens=32, num_pages=1)
    pages, dx, slots = kv.new_pages(), _dev(x), np.arange(6)
    kv.append(pages, k=dx[:3], v=dx[:3], slots=_dev(slots[:3]))
    kv.append(pages, k=dx[5:], v=dx[5:], slots=_dev(slots[5:]))
    torch.cuda.synchronize()
    kv.check()
    from shard_decomposed_gemm_amd import AgemmError
    for i in (3, 4):
        kv.append(pages, k=dx[i:i + 1], v=dx[i:i + 1], slots=_dev(slots[i:i + 1]))
        torch.cuda.synchronize()
        with pytest.raises(AgemmError, match="not finite or beyond"):
            kv.check()
        kv.check()  # cleared
    kn, ks, kb, vn, vs, vb = okv.unpack(pages.cpu().numpy(), 1, D, 32)
    on, os_, ob, _ = okv.quantise(x)
    for n, s, b in ((kn, ks, kb), (vn, vs, vb)):
        np.testing.assert_array_equal(s[:6], os_)
        np.testing.assert_array_equal(b[:6], ob)
        np.testing.assert_array_equal(n[:6], on)
        assert np.isfinite(okv.held(n[:6], s[:6], b[:6])).all()
        assert (okv.held(n[1], s[1], b[1]) == 0.625).all() and (okv.held(n[0], s[0], b[0]) == 0).all()


def test_append_reports_slots_and_positions_out_of_range():
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    T, Hq, Hkv, D, P = 4, 2, 1, 64, 2
    c = _append_case(5, T, Hq, Hkv, D, 64, False, False, length=100)
    kv = _cache(Hq, Hkv, D, page_tokens=32, num_pages=P)
    x, table = _dev(c["x"]), _dev(c["table"])
    q, k, v, eq, ek = _append_expected(c, Hq, Hkv)
    for slots, pos, match, left in (([0, 64, 2, -5], c["pos"], "slot 64 past", []),
                                    ([0, 1, 2, 3], [c["pos"][0], 100, c["pos"][2], -1], "outside the rotation table", [1, 3])):
        pages = kv.new_pages()
        q_out = torch.full((T, Hq, D), 3.0, dtype=torch.float16, device=gu.dev())
        kv.append(pages, q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], slots=_dev(np.array(slots)),
                  positions=_dev(np.array(pos)), rope=table, q_out=q_out)
        torch.cuda.synchronize()
        with pytest.raises(AgemmError, match=match):
            kv.check()
        got = q_out.cpu().numpy().astype(np.float64)
        for t in range(T):
            if t in left:
                assert (got[t] == 3).all()
            else:
                assert (np.abs(got[t] - q[t]) <= _half(np.abs(q[t]) + eq[t]) + 2 * eq[t]).all()
        kn, ks, *_ = okv.unpack(pages.cpu().numpy(), Hkv, D, 32)
        kept = [s for t, s in enumerate(slots) if 0 <= s < 64 and t not in left]
        assert (ks[kept] > 0).all() and (np.delete(ks, kept, 0) == 0).all() and (np.delete(kn, kept, 0) == 0).all()
    k_out, v_out = (torch.full((2, Hkv, D), 5.0, dtype=torch.float16, device=gu.dev()) for _ in range(2))
    kv.read(pages, _dev(np.array([64, -1])), k_out, v_out)
    torch.cuda.synchronize()
    with pytest.raises(AgemmError, match="past the last page"):
        kv.check()
    assert (k_out == 5).all() and (v_out == 5).all()


def test_append_slots_beyond_32_bit_offsets():
    """A cache of over 4 GiB: the last page's bytes lie beyond 2^32."""
    import torch
    D, page = 256, 256
    P = (1 << 32) // (page * (D + 8)) + 2
    kv = _cache(1, 1, D, page_tokens=page, num_pages=P)
    pages = torch.zeros(P, kv.page_bytes, dtype=torch.uint8, device=gu.dev())
    r = np.random.default_rng(1)
    x = r.standard_normal((3, 1, D)).astype(np.float16)
    slots = np.array([P * page - 1, 5, (P - 1) * page])
    kv.append(pages, k=_dev(x), v=_dev(x), slots=_dev(slots))
    last = okv.unpack(pages[-1:].cpu().numpy(), 1, D, page)
    _check_rows(x[[2, 0]].astype(np.float64), 0.0, *(y[[0, page - 1]] for y in last[:3]))
    table = torch.tensor([[P - 1, 0]], dtype=torch.int32, device=gu.dev())
    q = _dev(x[:1])
    out = torch.zeros(1, 1, D, dtype=torch.float32, device=gu.dev())
    lens = torch.tensor([1], dtype=torch.int32, device=gu.dev())
    kv.attend(pages, q, lens, table, out)
    torch.cuda.synchronize()
    kv.check()
    V = okv.held(*(y[0] for y in last[3:]))
    np.testing.assert_allclose(out.cpu().numpy()[0], V, rtol=2.0 ** -20)


# ---------------------------------------------------------------- attention

def _sequences(seed, Hkv, D, page, lens, garbage=True):
    """A cache of random tokens with shuffled pages: (pages, table, K, V of each sequence). Bytes of no sequence are
    all ones: NaN pairs."""
    r = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 1
    x = r.standard_normal((2, P * page, Hkv, D)) * np.exp(0.5 * r.standard_normal((2, 1, Hkv, D)))
    kn, ks, kb, _ = okv.quantise(x[0])
    vn, vs, vb, _ = okv.quantise(x[1])
    ids = r.permutation(P)
    table = np.full((len(lens), max(1, max(need))), -7, dtype=np.int32)  # nothing reads the rest
    used = np.zeros(P * page, dtype=bool)
    K, V = [], []
    at = 0
    for i, n in enumerate(lens):
        table[i, :need[i]] = ids[at:at + need[i]]
        slot = (table[i, :need[i], None].astype(int) * page + np.arange(page)).reshape(-1)[:n]
        at += need[i]
        used[slot] = True
        K.append(okv.held(kn[slot], ks[slot], kb[slot]))
        V.append(okv.held(vn[slot], vs[slot], vb[slot]))
    if garbage:
        nan = np.float16(np.nan)
        for n in (kn, vn):
            n[~used] = 15
        for y in (ks, kb, vs, vb):
            y[~used] = nan
    return okv.pack(kn, ks, kb, vn, vs, vb, page), table, K, V


def _check_attend(got, lse, q, K, V, seen, scale, f32):
    O, want, mass, reach = okv.attend(q, K, V, seen, scale)
    D, L = q.shape[-1], max(1, len(K))
    # scores: a dot product of D terms, the factor and the exponent's argument, each within 2^-24 of reach
    d = (reach * (D + 16) * 2.0 ** -24 + 2.0 ** -21)[..., None]
    # weights: the scores' error twice (also in the sum), their rounding to two or one binary16, L additions
    bound = mass * (2 * d + (2.0 ** -21 if f32 else 2.0 ** -11) + (L + 64) * 2.0 ** -24)
    bound = bound + (np.abs(O) * 2.0 ** -23 if f32 else _half(np.abs(O) + bound))
    assert (np.abs(got - O) <= bound).all(), (np.abs(got - O) / bound).max()
    assert (got[np.asarray(seen) <= 0] == 0).all()
    if lse is not None:
        some = np.asarray(seen) > 0
        assert (lse[~some] == np.float32(okv.LOWEST)).all()
        assert (np.abs(lse - want)[some] <= (2 * d[..., 0] + (L + 64) * 2.0 ** -24 + np.abs(want) * 2.0 ** -22)[some]).all()


def _run_attend(kv, pages, table, lens, q, starts=None, max_q=1, f32=True, q_off=None, causal=True, scale=None,
                with_lse=True, max_kv=None, workspace=None, stream=None):
    import torch
    T, Hq, D = q.shape[0], q.shape[1], q.shape[2]
    out = torch.full((T, Hq, D), 9.0, dtype=torch.float32 if f32 else torch.float16, device=gu.dev())
    lse = torch.full((T, Hq), 9.0, dtype=torch.float32, device=gu.dev()) if with_lse else None
    i32 = lambda x: None if x is None else _dev(np.asarray(x, dtype=np.int32))  # noqa: E731
    kv.attend(pages, q, i32(lens), i32(table), out, lse=lse, q_start=i32(starts), max_q=max_q, q_off=i32(q_off),
              causal=causal, scale=scale, max_kv=max_kv, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    kv.check()
    return out.cpu().numpy().astype(np.float64), None if lse is None else lse.cpu().numpy().astype(np.float64)


DECODES = [
    # Hq, Hkv, D, page, lens
    (8, 2, 128, 32, [1, 2, 31, 32, 33, 0, 63, 65, 127, 300]),
    (12, 1, 128, 64, [64, 129, 1000, 5]),
    (16, 1, 128, 64, [95, 96, 97]),
    (3, 3, 128, 128, [500, 128, 1]),
    (8, 1, 64, 32, [17, 0, 160, 1025]),
    (5, 5, 64, 256, [255, 256, 257]),
    (10, 2, 256, 64, [40, 333]),
    (1, 1, 256, 128, [1, 700]),
    (40, 2, 128, 64, [77, 515]),
    (72, 1, 64, 32, [200]),
    (64, 8, 128, 64, [2500]),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens", DECODES)
def test_attend_single_tokens(Hq, Hkv, D, page, lens, f32):
    print(f"[kv decode] {Hq} {Hkv} {D} {page} {lens} {f32}", flush=True)
    pages, table, K, V = _sequences(Hq + D, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = np.random.default_rng(2).standard_normal((len(lens), Hq, D)).astype(np.float16)
    got, lse = _run_attend(kv, _dev(pages), table, lens, _dev(q), f32=f32)
    for i, n in enumerate(lens):
        _check_attend(got[i:i + 1], lse[i:i + 1], q[i:i + 1], K[i], V[i], [n], D ** -0.5, f32)


QUERIES = [
    # Hq, Hkv, D, page, [(queries, length)], q_off, causal
    (8, 2, 128, 32, [(4, 100), (1, 33), (0, 50), (3, 3), (5, 2), (2, 0)], None, True),
    (16, 2, 64, 64, [(7, 200), (2, 64)], None, True),
    (4, 4, 256, 64, [(5, 70), (6, 6)], None, True),
    (6, 2, 128, 64, [(20, 150), (33, 33), (70, 95), (17, 5)], None, True),
    (2, 2, 64, 32, [(130, 130), (65, 300), (1, 9)], None, True),
    (3, 1, 256, 128, [(90, 128)], None, True),
    (8, 1, 128, 64, [(40, 333), (64, 64)], None, True),
    (4, 2, 128, 32, [(6, 60), (6, 60), (6, 60), (80, 40)], [-3, 100, -50, -10], True),  # another rank's keys
    (4, 2, 128, 32, [(6, 60), (3, 0), (50, 77)], None, False),
    (12, 1, 64, 32, [(30, 31), (29, 64)], [40, -20], True),
    (16, 1, 128, 64, [(150, 1000)], None, True),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,shape,q_off,causal", QUERIES)
def test_attend_several_queries(Hq, Hkv, D, page, shape, q_off, causal, f32):
    """Drafts and prompts: masks that leave rows empty, a strided q, rows behind the last sequence."""
    print(f"[kv queries] {Hq} {Hkv} {D} {page} {shape} {q_off} {causal} {f32}", flush=True)
    lens = [n for _, n in shape]
    starts = np.concatenate([[0], np.cumsum([q for q, _ in shape])])
    T = int(starts[-1]) + 3
    pages, table, K, V = _sequences(Hq + D, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    wide = _dev(np.random.default_rng(4).standard_normal((T, Hq + 2, D + 8)).astype(np.float16))
    q = wide[:, 1:-1, 8:]
    got, lse = _run_attend(kv, _dev(pages), table, lens, q, starts=starts, max_q=max(1, max(n for n, _ in shape)),
                           f32=f32, q_off=q_off, causal=causal, scale=0.11)
    hq = q.cpu().numpy()
    for i, (n, L) in enumerate(shape):
        off = L - n if q_off is None else q_off[i]
        seen = np.clip(off + np.arange(n) + 1, 0, L) if causal else np.full(n, L)
        rows = slice(starts[i], starts[i + 1])
        _check_attend(got[rows], lse[rows], hq[rows], K[i], V[i], seen, 0.11, f32)
    assert (got[starts[-1]:] == 9).all() and (lse[starts[-1]:] == 9).all()


LONG = [
    # Hq, Hkv, D, page, [(queries, length)], q_off, max_kv: items in several runs, joined
    (8, 1, 128, 64, [(40, 4200)], None, None),
    (4, 2, 64, 32, [(70, 3001), (3, 90), (0, 2000), (66, 66)], None, None),
    (3, 1, 256, 64, [(50, 2100), (17, 1030)], None, None),
    (2, 1, 128, 32, [(80, 2500), (80, 2500), (80, 40)], [1000, -79, -40], None),
    (16, 2, 128, 64, [(4, 3000), (2, 1500), (1, 2999)], [2000, -1, -5], None),
    (5, 1, 64, 32, [(3, 1100), (6, 4000), (0, 3000), (1, 0)], None, None),
    (4, 1, 128, 64, [(1, 9000), (1, 7), (1, 5000)], None, 64),       # longer than max_kv says
    (4, 1, 128, 64, [(1, 9000), (1, 7), (1, 20000)], None, 2048),
    (1, 1, 64, 256, [(1, 90000)], None, 3000),
    (8, 1, 128, 64, [(40, 9000)], None, 1200),
    (16, 1, 64, 128, [(1, 70000)], None, None),                      # as many runs as the join takes
    (2, 2, 64, 32, [(1, 70 * (i % 7 == 0) + i) for i in range(69)] + [(1, 6000)], None, None),
    (2, 1, 64, 32, [(1, 1400 if i == 200 else i % 9) for i in range(520)], None, None),
    (2, 1, 64, 32, [(1, 1400 if i == 500 else i % 9) for i in range(512)], None, None),
]


BATCHES = [  # many rows, the same columns: tiles of more than one group of 64 sequences, none of some, and 256-row tiles
    (4, 1, 64, 32, [(i * 37 % 71, i * 37 % 71 + i % 5) for i in range(130)], None, None),
    (2, 2, 128, 32, [(70 if i == 300 else i % 2, 80 if i == 300 else i % 40) for i in range(512)], None, None),
    (1, 1, 64, 32, [(90 if i in (3, 519) else i % 2, 95 if i in (3, 519) else i % 40) for i in range(520)], None, None),
    (8, 2, 128, 32, [({300: 333, 77: 90}.get(i, i % 3), {300: 350, 77: 60}.get(i, i % 40)) for i in range(512)], None, 4096),
    (8, 2, 128, 64, [({3: 200, 511: 130}.get(i, 0), 260 - i % 2) for i in range(512)],
     [-30 if i == 3 else 200 for i in range(512)], 2048),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,shape,q_off,max_kv", LONG + BATCHES)
def test_attend_joins_runs(Hq, Hkv, D, page, shape, q_off, max_kv, f32):
    print(f"[kv runs] {Hq} {Hkv} {D} {page} {shape[:4]} {len(shape)} {q_off} {max_kv} {f32}", flush=True)
    lens = [n for _, n in shape]
    starts = np.concatenate([[0], np.cumsum([q for q, _ in shape])])
    pages, table, K, V = _sequences(Hq + D, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = np.random.default_rng(4).standard_normal((int(starts[-1]), Hq, D)).astype(np.float16)
    got, lse = _run_attend(kv, _dev(pages), table, lens, _dev(q), starts=starts, max_q=max(n for n, _ in shape), f32=f32,
                           q_off=q_off, max_kv=max_kv, with_lse=f32)
    for i, (n, L) in enumerate(shape):
        off = L - n if q_off is None else q_off[i]
        rows = slice(starts[i], starts[i + 1])
        _check_attend(got[rows], None if lse is None else lse[rows], q[rows], K[i], V[i],
                      np.clip(off + np.arange(n) + 1, 0, L), D ** -0.5, f32)


@pytest.mark.parametrize("nq", [1, 3, 200])
def test_attend_large_scores_and_masked_extremes(nq):
    """Scores far apart (one key takes all the weight, the running maximum rises late), and values of the type's
    extremes in tokens that the mask hides."""
    D, page, L = 128, 64, 333
    r = np.random.default_rng(8)
    x = r.standard_normal((2, 384, 1, D))
    x[0, :L, 0] *= (1 + np.arange(L) % 97)[:, None] / 4  # growing keys
    x[1, 200:] = np.where(r.random((184, 1, D)) < 0.5, 20000, -20000)  # hidden from the first rows
    kn, ks, kb, _ = okv.quantise(x[0])
    vn, vs, vb, _ = okv.quantise(x[1])
    pages = okv.pack(kn, ks, kb, vn, vs, vb, page)
    kv = _cache(1, 1, D, page_tokens=page, num_pages=6)
    q = 3 * r.standard_normal((nq, 1, D)).astype(np.float16)
    off = [199 - nq]
    got, lse = _run_attend(kv, _dev(pages), np.arange(6)[None], [L], _dev(q), starts=[0, nq], max_q=nq, q_off=off)
    seen = off[0] + 1 + np.arange(nq)
    _check_attend(got, lse, q, okv.held(kn, ks, kb)[:L], okv.held(vn, vs, vb)[:L], seen, D ** -0.5, True)


def test_attend_shared_pages_and_table_row():
    """Sequences on the same pages (a shared prefix) through one table row with stride 0."""
    import torch
    Hq, Hkv, D, page = 4, 2, 64, 32
    pages, table, K, V = _sequences(9, Hkv, D, page, [200])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = np.random.default_rng(3).standard_normal((5, Hq, D)).astype(np.float16)
    lens = np.array([1, 50, 64, 199, 200], dtype=np.int32)
    shared = _dev(table).expand(5, -1)
    assert shared.stride(0) == 0
    out = torch.zeros(5, Hq, D, device=gu.dev())
    kv.attend(_dev(pages), _dev(q), _dev(lens), shared, out)
    torch.cuda.synchronize()
    kv.check()
    for i, n in enumerate(lens):
        _check_attend(out[i:i + 1].cpu().numpy().astype(np.float64), None, q[i:i + 1], K[0], V[0], [n], D ** -0.5, True)


@pytest.mark.parametrize("nq", [1, 40])
def test_attend_reports_what_it_cannot_use(nq):
    """Page ids outside the cache, lengths outside the table, rows outside q: reported, and nothing else touched."""
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    Hq, Hkv, D, page = 4, 2, 128, 32
    pages, table, K, V = _sequences(11, Hkv, D, page, [96, 96])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    dp = _dev(pages)
    q = np.random.default_rng(3).standard_normal((2 * nq, Hq, D)).astype(np.float16)
    base = dict(lens=[96, 96], table=table, starts=[0, nq, 2 * nq], max_q=nq)

    def run(match, **change):
        a = {**base, **change}
        out = torch.full((2 * nq, Hq, D), 9.0, device=gu.dev())
        i32 = lambda x: _dev(np.asarray(x, dtype=np.int32))  # noqa: E731
        kv.attend(dp, _dev(q), i32(a["lens"]), i32(a["table"]), out, q_start=i32(a["starts"]), max_q=a["max_q"])
        torch.cuda.synchronize()
        with pytest.raises(AgemmError, match=match):
            kv.check()
        return out.cpu().numpy().astype(np.float64)

    def good(got, i, keys=slice(None), seen=None):
        rows = slice(i * nq, (i + 1) * nq)
        _check_attend(got[rows], None, q[rows], K[i][keys], V[i][keys], 96 - nq + 1 + np.arange(nq) if seen is None
                      else seen, D ** -0.5, True)

    for bad in (pages.shape[0], -1, 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[1, 0] = bad  # the first 32 tokens of sequence 1 count as not seen
        got = run("page id", table=t)
        good(got, 0)
        good(got, 1, slice(32, None), np.maximum(0, 96 - nq + 1 + np.arange(nq) - 32))
    for bad, seen in ((97, None), (2 ** 31 - 1, None), (-1, np.zeros(nq)), (-2 ** 31, np.zeros(nq))):
        got = run("length", lens=[96, bad])
        good(got, 0)
        good(got, 1, seen=seen)
    got = run("query rows", starts=[0, nq, 2 * nq + 1], max_q=nq + 1)  # rows past q
    good(got, 0)
    assert (got[nq:] == 9).all()
    got = run("query rows", starts=[-1, nq, 2 * nq], max_q=nq + 1)
    assert (got[:nq] == 9).all()
    got = run("query rows", starts=[nq, 0, nq])
    assert (got[nq:] == 9).all()  # sequence 0 has a negative number of rows, sequence 1 the first ones
    if nq > 1:
        got = run("query rows", max_q=nq - 1)
        assert (got == 9).all()


def test_attend_same_bits_every_time_and_on_another_stream():
    import torch
    Hq, Hkv, D, page = 16, 2, 128, 64
    lens = [3000, 17, 800]
    pages, table, K, V = _sequences(21, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = _dev(np.random.default_rng(3).standard_normal((3, Hq, D)).astype(np.float16))
    dp = _dev(pages)
    torch.cuda.synchronize()
    first, lse = _run_attend(kv, dp, table, lens, q)
    other = torch.cuda.Stream()
    ws = kv.workspace(3, 1, 4096)
    for stream, w in ((None, None), (other, None), (None, ws), (other, ws)):
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        # the work-split follows max_kv, which both calls leave at the table's width
        again, lse2 = _run_attend(kv, dp, table, lens, q, stream=stream, workspace=w)
        np.testing.assert_array_equal(first, again)
        np.testing.assert_array_equal(lse, lse2)


def test_two_calls_at_once_on_two_streams():
    """Two attention calls and an append in flight together, each with its own workspace."""
    import torch
    Hq, Hkv, D, page = 8, 2, 128, 64
    lens = [4000, 900]
    pages, table, K, V = _sequences(22, Hkv, D, page, lens)
    P = pages.shape[0]
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=P)
    dp = _dev(pages)
    dl, dt = _dev(np.array(lens, dtype=np.int32)), _dev(table)
    qs = [_dev(np.random.default_rng(s).standard_normal((2, Hq, D)).astype(np.float16)) for s in (1, 2)]
    outs = [torch.zeros(2, Hq, D, device=gu.dev()) for _ in range(2)]
    spare = (set(range(P)) - set(table.reshape(-1).tolist())).pop()
    kx = torch.randn(16, Hkv, D, device=gu.dev()).half()
    slots = _dev(spare * page + np.arange(16))
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [kv.workspace(2, 1, 4096) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s in (0, 1):
            kv.attend(dp, qs[s], dl, dt, outs[s], workspace=ws[s], stream=streams[s])
        kv.append(dp, k=kx, v=kx, slots=slots, stream=streams[2])
    torch.cuda.synchronize()
    kv.check()
    for s in (0, 1):
        for i, n in enumerate(lens):
            _check_attend(outs[s][i:i + 1].cpu().numpy().astype(np.float64), None, qs[s][i:i + 1].cpu().numpy(), K[i],
                          V[i], [n], D ** -0.5, True)


def test_decode_step_in_a_graph():
    """A captured step - append the token, attend over the cache with it - replayed with new inputs, lengths and
    slots in the same tensors: every replay equals the eager calls."""
    import torch
    Hq, Hkv, D, page, B = 8, 2, 128, 32, 3
    pages, table, K, V = _sequences(31, Hkv, D, page, [128, 64, 96])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    rope = _dev(_table(200, D))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.float16, device=gu.dev())
    pos = torch.zeros(B, dtype=torch.int64, device=gu.dev())
    slots, lens, dt = torch.zeros_like(pos), torch.zeros(B, dtype=torch.int32, device=gu.dev()), _dev(table)
    qr = torch.zeros(B, Hq, D, dtype=torch.float16, device=gu.dev())
    out, lse = torch.zeros(B, Hq, D, device=gu.dev()), torch.zeros(B, Hq, device=gu.dev())
    dp = _dev(pages)
    ws = kv.workspace(B, 1, 128)

    def step(p, o, z, w):
        kv.append(p, q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], slots=slots, positions=pos, rope=rope, q_out=qr)
        kv.attend(p, qr, lens, dt, o, lse=z, max_kv=128, workspace=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(dp.clone(), out, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(dp, out, lse, ws)
    eager_pages, eo, ez = dp.clone(), torch.zeros_like(out), torch.zeros_like(lse)
    for n in ([128, 3, 60], [1, 64, 33], [70, 32, 96], [128, 64, 96]):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        at = torch.tensor(n, device=gu.dev())
        lens.copy_(at)
        pos.copy_(at - 1)
        slots.copy_(dt.long().gather(1, ((at - 1) // page)[:, None])[:, 0] * page + (at - 1) % page)
        graph.replay()
        torch.cuda.synchronize()
        step(eager_pages, eo, ez, None)
        torch.cuda.synchronize()
        kv.check()
        assert torch.equal(out, eo) and torch.equal(lse, ez) and torch.equal(dp, eager_pages)


@pytest.mark.parametrize("nq", [1, 40])
def test_joined_runs_in_a_graph(nq):
    """Attention over long sequences, captured once; replays with other lengths equal the eager calls, and what lies in
    the workspace before a replay does not matter."""
    import torch
    Hq, Hkv, D, page, B = 8, 2, 64, 64, 3
    pages, table, K, V = _sequences(33, Hkv, D, page, [4000, 2600, 1500])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    dp, dt = _dev(pages), _dev(table)
    q = _dev(np.random.default_rng(6).standard_normal((B * nq, Hq, D)).astype(np.float16))
    starts, lens = _dev(np.arange(B + 1, dtype=np.int32) * nq), torch.zeros(B, dtype=torch.int32, device=gu.dev())
    out, eo = (torch.zeros(B * nq, Hq, D, device=gu.dev()) for _ in range(2))
    ws = kv.workspace(B, nq, 4000)
    assert ws.numel() > 0

    def step(o, w):
        kv.attend(dp, q, lens, dt, o, q_start=starts, max_q=nq, max_kv=4000, workspace=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, ws)
    for n in ([4000, 2600, 1500], [1, 2600, 0], [nq, 0, 1500], [3999, 33, 700], [4000, 2600, 1500]):
        lens.copy_(torch.tensor(n))
        ws.fill_(0xFF)
        out.fill_(9)
        eo.fill_(9)
        graph.replay()
        step(eo, None)
        torch.cuda.synchronize()
        kv.check()
        assert torch.equal(out, eo)
    hq = q.cpu().numpy()
    for i, L in enumerate(n):
        rows = slice(i * nq, (i + 1) * nq)
        _check_attend(out[rows].cpu().numpy().astype(np.float64), None, hq[rows], K[i], V[i],
                      np.clip(L - nq + 1 + np.arange(nq), 0, L), D ** -0.5, True)


def test_ranks_append_attend_and_combine():
    """Flash Decode over W shards of the cache, all of it through this library: append each rank's share of a
    sequence's tokens, attend over it, combine the partials. One rank holds nothing of one sequence."""
    import torch
    from shard_decomposed_gemm_amd import FdCombine
    W, Hq, Hkv, D, page, B, L = 4, 16, 4, 128, 32, 2, 150
    r = np.random.default_rng(17)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=16)
    table = _table(L + 1, D)
    qkv = r.standard_normal((B, L, Hq + 2 * Hkv, D)).astype(np.float16)
    share = [[60, 30, 60, 0], [1, 64, 33, 52]]  # tokens of each rank, in order
    o_parts, lse_parts, Ks, Vs = [], [], [[], []], [[], []]
    rope = _dev(table)
    for w in range(W):
        pages = kv.new_pages()
        ids = r.permutation(16)[:8].reshape(B, 4).astype(np.int32)
        lens = np.array([share[b][w] for b in range(B)], dtype=np.int32)
        q_rot = torch.zeros(B, Hq, D, dtype=torch.float16, device=gu.dev())
        for b in range(B):
            first = sum(share[b][:w])
            # every rank walks all tokens; slots of other ranks' tokens are negative
            slots = np.full(L, -1)
            mine = np.arange(share[b][w])
            slots[first + mine] = ids[b, mine // page] * page + mine % page
            x = _dev(qkv[b])
            qo = torch.zeros(L, Hq, D, dtype=torch.float16, device=gu.dev())
            kv.append(pages, q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], slots=_dev(slots),
                      positions=_dev(np.arange(L)), rope=rope, q_out=qo)
            q_rot[b] = qo[-1]
            if len(mine):
                k_out, v_out = (torch.zeros(len(mine), Hkv, D, dtype=torch.float16, device=gu.dev()) for _ in range(2))
                kv.read(pages, _dev(slots[first + mine]), k_out, v_out)
                Ks[b].append(k_out.cpu().numpy())
                Vs[b].append(v_out.cpu().numpy())
        out = torch.full((B, Hq, D), float("nan"), device=gu.dev())
        lse = torch.full((B, Hq), float("nan"), device=gu.dev())
        kv.attend(pages, q_rot, _dev(lens), _dev(ids), out, lse=lse)
        o_parts.append(out.view(B * Hq, D))
        lse_parts.append(lse.view(B * Hq))
    kv.check()
    fdc = FdCombine(W, B * Hq, D, heads_per_tile=8, out_dtype="f32")
    O = torch.full((B * Hq, D), float("nan"), device=gu.dev())
    sp, sc = fdc.streams()
    torch.cuda.synchronize()
    fdc.produce(o_parts, lse_parts, stream=sp)
    fdc.run_fused(O, stream=sc)
    torch.cuda.synchronize()
    fdc.check()
    got = O.cpu().numpy().astype(np.float64).reshape(B, Hq, D)
    q = q_rot.cpu().numpy()
    for b in range(B):
        K, V = np.concatenate(Ks[b]), np.concatenate(Vs[b])
        want, _, mass, reach = okv.attend(q[b:b + 1], K, V, [L], D ** -0.5)
        d = (reach * (D + 16) * 2.0 ** -24 + 2.0 ** -21)[..., None]
        bound = mass * (4 * d + (L + 64) * 2.0 ** -24) + fdo.tolerance("f32") * np.abs(V).max()
        assert (np.abs(got[b] - want[0]) <= bound[0]).all()


def test_binding_refuses_wrong_tensors():
    import torch
    Hq, Hkv, D = 4, 2, 64
    kv = _cache(Hq, Hkv, D, page_tokens=32, num_pages=2)
    pages = kv.new_pages()
    q = torch.zeros(3, Hq, D, dtype=torch.float16, device=gu.dev())
    k = torch.zeros(3, Hkv, D, dtype=torch.float16, device=gu.dev())
    slots = torch.zeros(3, dtype=torch.int64, device=gu.dev())
    lens, table = torch.ones(3, dtype=torch.int32, device=gu.dev()), torch.zeros(3, 1, dtype=torch.int32, device=gu.dev())
    out = torch.zeros(3, Hq, D, device=gu.dev())
    from shard_decomposed_gemm_amd import AgemmError
    for err, call in [
        (ValueError, lambda: kv.append(pages)),
        (TypeError, lambda: kv.append(pages, k=k.float(), v=k, slots=slots)),
        (TypeError, lambda: kv.append(pages, k=k.cpu(), v=k, slots=slots)),
        (ValueError, lambda: kv.append(pages, k=k[:, :1], v=k, slots=slots)),
        (ValueError, lambda: kv.append(pages, k=k, v=k, slots=slots[:2])),
        (TypeError, lambda: kv.append(pages, k=k, v=k, slots=slots.int())),
        (ValueError, lambda: kv.append(pages[:1], k=k, v=k, slots=slots)),
        (ValueError, lambda: kv.append(pages, k=k.transpose(0, 2), v=k, slots=slots)),
        (AgemmError, lambda: kv.append(pages, k=k, slots=slots)),
        (AgemmError, lambda: kv.append(pages, q=q)),
        (AgemmError, lambda: kv.append(pages, q=q, q_out=q[:1].expand(3, Hq, D))),
        (AgemmError, lambda: kv.append(None, k=k, v=k, slots=slots)),
        (TypeError, lambda: kv.attend(pages, q.float(), lens, table, out)),
        (ValueError, lambda: kv.attend(pages, q, lens, table[:2], out)),
        (TypeError, lambda: kv.attend(pages, q, lens, table.long(), out)),
        (TypeError, lambda: kv.attend(pages, q, lens.long(), table, out)),
        (ValueError, lambda: kv.attend(pages, q, lens, table, out[:2])),
        (TypeError, lambda: kv.attend(pages, q, lens, table, out.double())),
        (ValueError, lambda: kv.attend(pages, q, lens, table, out, lse=torch.zeros(3, Hq + 1, device=gu.dev()))),
        (TypeError, lambda: kv.attend(pages, q, lens, table, out, workspace=torch.zeros(16, device=gu.dev()))),
        (AgemmError, lambda: kv.attend(pages, q, lens, table, out, max_q=2)),
        (AgemmError, lambda: kv.attend(pages, q, lens, table, out, scale=float("nan"))),
        (ValueError, lambda: kv.read(pages, slots, k, k[:2])),
        (TypeError, lambda: kv.read(pages, slots.int(), k, k)),
    ]:
        with pytest.raises(err):
            call()
    kv.attend(pages, q[:0], lens[:0], table[:0], out[:0])  # nothing
    torch.cuda.synchronize()
    kv.check()
