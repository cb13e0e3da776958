"""GPU tests of a step with drafted tokens on the key/value cache (include/kvcache.h) against the binary64 oracle.

Tolerances count roundings as tests/test_gpu_kv.py does; whole numbers and moved bits have to be equal.
"""
import numpy as np
import pytest

from oracle import kv as okv
from oracle import kvtree as okt
from tests import gpu_util as gu
from tests.test_gpu_kv import _cache, _dev, _half, _sequences

pytestmark = pytest.mark.gpu

PAD = 77  # fills what a call must leave


def _i32(x):
    return None if x is None else _dev(np.asarray(x, dtype=np.int32))


def _full(shape, dtype, value=PAD):
    import torch
    return torch.full(shape, value, dtype=getattr(torch, dtype), device=gu.dev())


def _parents(r, n, kind="mixed"):
    """Trees whose parents come first."""
    if kind == "chain":
        return [-1] + list(range(n - 1)) if n else []
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    return [-1] + [int(i - 1) if r.random() < 0.4 else int(r.integers(0, i)) for i in range(1, n)] if n else []


def _starts(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


# ---------------------------------------------------------------- layout

TREES = [
    # sizes, words, kind, page, lengths before, rows before and behind
    ([1], 1, "mixed", 64, [0], 0, 0),
    ([8], 1, "mixed", 32, [777], 0, 5),
    ([64, 1, 0, 63], 1, "mixed", 32, [31, 0, 5, 64], 2, 70),
    ([64], 1, "chain", 256, [1000], 0, 0),
    ([65, 3, 128], 2, "mixed", 64, [100, 200, 1], 0, 1),
    ([200, 0, 77, 256], 4, "mixed", 128, [5, 6, 7, 8], 1, 0),
    ([256], 4, "chain", 32, [33], 0, 0),
    ([130, 192], 3, "star", 32, [0, 1], 0, 3),
    ([1024], 16, "chain", 64, [12345], 0, 0),
    ([1000, 1, 513], 16, "mixed", 64, [1, 2, 3], 3, 3),
    ([300, 320], 5, "star", 256, [1, 2], 0, 0),
    ([i % 9 for i in range(300)], 1, "mixed", 32, [i * 7 % 500 for i in range(300)], 0, 900),
]


def _tree_problem(seed, sizes, words, kind, page, lens, before=0, behind=0):
    r = np.random.default_rng(seed)
    parents = [_parents(r, n, kind) for n in sizes]
    T = before + sum(sizes) + behind
    parent = np.full(T, -5, dtype=np.int32)
    starts = _starts(sizes, before)
    width = max(1, max(-(-(n + m) // page) for n, m in zip(lens, sizes)))
    P = len(sizes) * width + 3
    table = r.permutation(P)[:len(sizes) * width].reshape(len(sizes), width).astype(np.int32)
    mask, pos, slots = np.zeros((T, words), dtype=np.uint64), np.zeros(T, dtype=np.int64), np.full(T, -1, dtype=np.int64)
    for b, n in enumerate(sizes):
        rows = slice(starts[b], starts[b + 1])
        parent[rows] = parents[b]
        mask[rows] = okt.masks(parents[b], words)
        pos[rows] = [lens[b] + len(a) - 1 for a in okt.ancestors(parents[b])]
        at = lens[b] + np.arange(n)
        slots[rows] = table[b, at // page].astype(np.int64) * page + at % page
    return dict(T=T, parent=parent, starts=starts, table=table, P=P, mask=mask, pos=pos, slots=slots,
                total=np.array(lens) + np.array(sizes))


def _run_tree(kv, c, lens, words, max_q=None, stream=None, **change):
    """The four outputs as numpy arrays."""
    import torch
    a = dict(parent=c["parent"], starts=c["starts"], table=c["table"], lens=lens)
    a.update(change)
    T, B = len(a["parent"]), len(a["lens"])
    mask, pos, slots, total = _full((T, words), "int64"), _full((T,), "int64"), _full((T,), "int64"), _full((B,), "int32")
    args = [_i32(a[k]) for k in ("parent", "starts", "lens", "table")]
    torch.cuda.synchronize()
    kv.tree(args[0], args[1], args[2], args[3], max_q or 64 * words, mask, positions=pos, slots=slots, total_len=total,
            stream=stream)
    torch.cuda.synchronize()
    return mask.cpu().numpy().view(np.uint64), pos.cpu().numpy(), slots.cpu().numpy(), total.cpu().numpy()


@pytest.mark.parametrize("sizes,words,kind,page,lens,before,behind", TREES)
def test_tree_against_the_oracle(sizes, words, kind, page, lens, before, behind):
    print(f"[kv tree] {sizes[:5]} {len(sizes)} {words} {kind} {page}", flush=True)
    c = _tree_problem(len(sizes) + words, sizes, words, kind, page, lens, before, behind)
    kv = _cache(1, 1, 64, page_tokens=page, num_pages=c["P"])
    got = _run_tree(kv, c, lens, words, max_q=max(sizes))
    kv.check()
    for g, k in zip(got, ("mask", "pos", "slots", "total")):
        np.testing.assert_array_equal(g, c[k])


def test_tree_optional_outputs_shared_table_and_nothing():
    import torch
    c = _tree_problem(3, [5, 9], 1, "mixed", 32, [3, 40])
    kv = _cache(1, 1, 64, page_tokens=32, num_pages=c["P"])
    parent, starts, lens = _i32(c["parent"]), _i32(c["starts"]), _i32([3, 40])
    mask = _full((14, 1), "int64")
    kv.tree(parent, starts, lens, None, 9, mask)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(mask.cpu().numpy().view(np.uint64), c["mask"])
    slots = _full((14,), "int64")
    row = _i32(c["table"][:1]).expand(2, -1)
    kv.tree(parent, starts, lens, row, 9, mask, slots=slots)
    torch.cuda.synchronize()
    at = np.concatenate([3 + np.arange(5), 40 + np.arange(9)])
    np.testing.assert_array_equal(slots.cpu().numpy(), c["table"][0, at // 32] * 32 + at % 32)
    kv.tree(parent[:0], starts[:1], lens[:0], row[:0], 9, mask[:0])  # nothing
    total = _full((2,), "int32")
    kv.tree(parent[:0], _i32([0, 0, 0]), lens, row, 9, mask[:0], slots=slots[:0], total_len=total)  # no nodes
    kv.tree(parent, starts[:1], lens[:0], row[:0], 9, mask, slots=slots)  # no sequences: padding alone
    torch.cuda.synchronize()
    kv.check()
    assert total.tolist() == [3, 40] and (slots == -1).all() and (mask == 0).all()


def test_tree_reports_what_it_cannot_use():
    from shard_decomposed_gemm_amd import AgemmError
    sizes, lens = [6, 7, 5], [10, 20, 30]
    c = _tree_problem(4, sizes, 1, "mixed", 32, lens, 0, 4)
    kv = _cache(1, 1, 64, page_tokens=32, num_pages=c["P"])
    width = c["table"].shape[1]

    def run(match, **change):
        got = _run_tree(kv, c, change.pop("lens", lens), 1, **change)
        with pytest.raises(AgemmError, match=match):
            kv.check()
        kv.check()
        return got

    def same(got, but=()):
        for b in range(3):
            rows = slice(c["starts"][b], c["starts"][b + 1])
            for g, k in zip(got[:3], ("mask", "pos", "slots")):
                if b not in but:
                    np.testing.assert_array_equal(g[rows], c[k][rows])
                elif k == "slots":
                    assert (g[rows] == -1).all()
                else:
                    assert (g[rows] == 0).all()
            assert got[3][b] == (lens[b] if b in but else c["total"][b])

    for bad in (6, 100, -2, -2 ** 31, 2 ** 31 - 1):  # taken as -1
        parent = c["parent"].copy()
        parent[4] = bad
        got = run("parent", parent=parent)
        assert got[0][4] == 1 << 4 and got[1][4] == 10
    for bad in (c["P"], -1, 2 ** 31 - 1, -2 ** 31):
        t = c["table"].copy()
        t[0, 0] = bad
        got = run("page id", table=t)
        assert (got[2][:6] == -1).all()
        np.testing.assert_array_equal(got[0], c["mask"])
        np.testing.assert_array_equal(got[1], c["pos"])
        np.testing.assert_array_equal(got[2][6:], c["slots"][6:])
    for bad in (-1, -2 ** 31, 2 ** 31 - 1, 32 * width - 6):
        got = run("length", lens=[10, bad, 30])
        assert got[3][1] == bad
        got[3][1] = 20
        same(got, but=[1])
    _run_tree(kv, c, [10, 32 * width - 7, 30], 1)  # just fits
    kv.check()
    got = run("query rows", max_q=6)
    same(got, but=[1])
    got = run("query rows", starts=[0, 6, 13, 23], parent=c["parent"])  # past T
    assert (got[2][13:] == -1).all() and got[3].tolist() == [16, 27, 30]
    got = run("query rows", starts=[0, 6, 4, 18], parent=np.full(22, -1))
    assert got[3].tolist()[:2] == [16, 20]
    got = run("query rows", starts=[-1, 6, 13, 18])
    assert (got[2][:6] == -1).all()


# ---------------------------------------------------------------- attention

def _check_rows(got, lse, q, K, V, seen, scale, f32):
    O, want, mass, reach = okt.attend(q, K, V, seen, scale)
    D, L = q.shape[-1], max(1, len(K))
    # as tests/test_gpu_kv.py counts: scores, weights and their sums
    d = (reach * (D + 16) * 2.0 ** -24 + 2.0 ** -21)[..., None]
    bound = mass * (2 * d + (2.0 ** -21 if f32 else 2.0 ** -11) + (L + 64) * 2.0 ** -24)
    bound = bound + (np.abs(O) * 2.0 ** -23 if f32 else _half(np.abs(O) + bound))
    assert (np.abs(got - O) <= bound).all(), (np.abs(got - O) / np.maximum(bound, 1e-300)).max()
    some = seen.any(-1)
    assert (got[~some] == 0).all()
    if lse is not None:
        assert (lse[~some] == np.float32(okv.LOWEST)).all()
        assert (np.abs(lse - want)[some] <= (2 * d[..., 0] + (L + 64) * 2.0 ** -24 + np.abs(want) * 2.0 ** -22)[some]).all()


def _run_attend(kv, pages, table, lens, q, starts, max_q, mask, f32=True, q_off=None, scale=None, max_kv=None,
                with_lse=True, workspace=None, stream=None):
    import torch
    T, Hq, D = q.shape
    out = _full((T, Hq, D), "float32" if f32 else "float16")
    lse = _full((T, Hq), "float32") if with_lse else None
    args = [_i32(x) for x in (lens, table, starts, q_off)]
    dm = _dev(mask.view(np.int64))
    torch.cuda.synchronize()
    kv.attend(pages, q, args[0], args[1], out, lse=lse, q_start=args[2], max_q=max_q, q_off=args[3], scale=scale,
              max_kv=max_kv, workspace=workspace, stream=stream, tree=dm)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), None if lse is None else lse.cpu().numpy().astype(np.float64)


ATTENDS = [
    # Hq, Hkv, D, page, [(queries, length)], words, kind, off: "last" (the tree's nodes are the last tokens), or a list
    (8, 2, 128, 32, [(4, 100), (1, 1), (3, 33), (2, 2), (0, 10), (4, 64)], 1, "mixed", None),
    (8, 1, 128, 64, [(2, 777)], 1, "chain", None),
    (16, 1, 128, 64, [(2, 300), (1, 31)], 1, "star", None),
    (4, 4, 256, 32, [(13, 150), (16, 16)], 1, "mixed", None),
    (3, 1, 256, 64, [(30, 400), (5, 5)], 1, "mixed", None),
    (2, 2, 64, 32, [(32, 95), (17, 65)], 1, "mixed", None),
    (32, 4, 64, 32, [(25, 500), (25, 26), (25, 25), (9, 700)], 1, "mixed", None),
    (8, 8, 64, 256, [(64, 64), (64, 200), (63, 90)], 1, "mixed", None),
    (64, 8, 128, 64, [(13, 790)], 1, "mixed", None),
    (8, 1, 128, 64, [(40, 333), (64, 1500)], 1, "chain", None),
    (6, 2, 128, 32, [(70, 150), (128, 300), (65, 65)], 2, "mixed", None),
    (5, 5, 128, 128, [(130, 200), (1, 4)], 3, "mixed", None),
    (2, 1, 64, 32, [(300, 700)], 5, "mixed", None),
    (1, 1, 128, 32, [(31, 31), (20, 2000)], 16, "mixed", None),
    (4, 2, 128, 32, [(5, 90), (8, 200), (3, 70)], 1, "mixed", [60, 170, 69]),        # the last level of a larger tree
    (8, 2, 128, 64, [(30, 300), (20, 100)], 2, "mixed", [200, 40]),
    (4, 2, 128, 32, [(6, 60), (6, 60), (6, 60), (40, 60)], 1, "mixed", [-3, 100, -70, -64]),  # rows that see nothing
    (4, 2, 64, 32, [(6, 300), (40, 300)], 1, "mixed", [3, 40]),                       # cached tokens past the tree's 64
    (16, 2, 64, 64, [(3, 3000), (2, 1500), (1, 2999)], 1, "mixed", None),             # joined runs, few rows
    (8, 1, 128, 64, [(40, 4200), (5, 5)], 1, "mixed", None),                          # joined runs, many rows
    (3, 1, 256, 64, [(50, 2100)], 1, "mixed", None),
    (24, 2, 128, 64, [(33, 2000)], 1, "mixed", None),
]


def _row_masks(r, n, words, kind, off):
    """Masks of n queries: of a tree's nodes, or (off given) of any nodes, some of none."""
    if off is None:
        return okt.masks(_parents(r, n, kind), words)
    m = r.integers(0, 2 ** 63, (n, words), dtype=np.uint64) & r.integers(0, 2 ** 63, (n, words), dtype=np.uint64)
    m |= r.integers(0, 2, (n, words), dtype=np.uint64) << np.uint64(63)
    m[r.random(n) < 0.2] = 0
    return m


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,shape,words,kind,q_off", ATTENDS)
def test_attend_a_tree(Hq, Hkv, D, page, shape, words, kind, q_off, f32):
    """Masks that leave rows empty, a strided q, rows behind the last sequence."""
    print(f"[kv attend tree] {Hq} {Hkv} {D} {page} {shape} {words} {kind} {q_off} {f32}", flush=True)
    r = np.random.default_rng(Hq + D + len(shape))
    lens = [n for _, n in shape]
    starts = _starts([n for n, _ in shape])
    T = int(starts[-1]) + 3
    pages, table, K, V = _sequences(Hq + D, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    mask = np.zeros((T, words), dtype=np.uint64)
    offs = [L - n for n, L in shape] if q_off is None else q_off
    for b, (n, L) in enumerate(shape):
        mask[starts[b]:starts[b + 1]] = _row_masks(r, n, words, kind, q_off)
    wide = _dev(r.standard_normal((T, Hq + 2, D + 8)).astype(np.float16))
    q = wide[:, 1:-1, 8:]
    got, lse = _run_attend(kv, _dev(pages), table, lens, q, starts, max(1, max(n for n, _ in shape)), mask, f32=f32,
                           q_off=q_off, scale=0.11)
    kv.check()
    hq = q.cpu().numpy()
    for b, (n, L) in enumerate(shape):
        rows = slice(starts[b], starts[b + 1])
        _check_rows(got[rows], lse[rows], hq[rows], K[b], V[b], okt.visible(mask[rows], offs[b], L), 0.11, f32)
    assert (got[starts[-1]:] == PAD).all() and (lse[starts[-1]:] == PAD).all()


def _batch(b, n, L):
    """b sequences of up to n queries and L tokens, the first of most."""
    return [(n - i % 3 if n > 3 else n, L - 37 * i % (L // 2)) for i in range(b)]


FORMS = [
    # Hq, Hkv, D, page, [(queries, length)], max_kv: every kernel, one run an item and several, joined by rows and by
    # workgroups (tests/test_kv_tree_host.py sees to it), a batch of more sequences than lengths are looked through,
    # lengths that max_kv does not say
    (32, 8, 128, 32, _batch(12, 25, 64), None),
    (2, 1, 128, 64, [(1, 60)], None),
    (2, 1, 128, 64, [(1, 2100)], None),
    (16, 2, 128, 64, _batch(6, 5, 2100), None),
    (16, 8, 128, 64, _batch(32, 40, 500), 500),
    (32, 8, 128, 64, _batch(32, 25, 1100), 1100),
    (16, 4, 128, 64, _batch(2, 32, 4000), None),
    (16, 8, 128, 64, _batch(16, 60, 200), None),
    (8, 8, 128, 64, _batch(16, 40, 2100), None),
    (32, 8, 256, 32, _batch(12, 25, 64), None),
    (32, 8, 256, 64, _batch(32, 25, 1100), 1100),
    (16, 8, 256, 32, _batch(12, 25, 64), None),
    (4, 4, 256, 64, _batch(12, 20, 4000), None),
    (1, 1, 256, 32, [(1, 64)], None),
    (1, 1, 256, 64, [(1, 2100)], None),
    (8, 1, 256, 64, _batch(12, 5, 2100), None),
    (2, 1, 64, 32, [(20, 64)], None),
    (32, 8, 64, 64, _batch(32, 25, 1100), 1100),
    (4, 1, 64, 32, [(1, 64)], None),
    (4, 1, 64, 32, [(1, 2100)], None),
    (32, 4, 64, 32, _batch(3, 5, 2100), None),
    (16, 8, 64, 64, _batch(12, 60, 200), None),
    (8, 1, 64, 64, _batch(4, 48, 2100), None),
    (16, 8, 64, 64, _batch(32, 25, 500), 500),
    (8, 8, 64, 64, _batch(32, 40, 2100), None),
    (8, 1, 128, 64, [(4, 9000)], 1300),
    (8, 1, 64, 32, [(4, 9000), (3, 100), (4, 5000)], 3000),
    (8, 2, 128, 64, [(13, 3000), (16, 20), (0, 900), (5, 2000)], 5000),
    (16, 2, 128, 64, [(64, 6000)], 1100),
    (4, 4, 128, 32, [(i % 3, i % 3 + 1400 if i == 300 else i % 40 + 3) for i in range(520)], 1400),
    (2, 1, 128, 32, [(40 if i == 70 else i % 4, 1500 if i in (3, 70) else i % 90 + 40) for i in range(130)], 1500),
    (8, 1, 64, 32, [(i % 9, 60 * i + 9) for i in range(70)], None),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,shape,max_kv", FORMS)
def test_attend_a_tree_in_every_form(Hq, Hkv, D, page, shape, max_kv, f32):
    print(f"[kv tree forms] {Hq} {Hkv} {D} {page} {shape[:4]} {len(shape)} {max_kv} {f32}", flush=True)
    r = np.random.default_rng(len(shape) + D)
    lens = [n for _, n in shape]
    starts = _starts([n for n, _ in shape])
    pages, table, K, V = _sequences(Hq + D, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    mask = np.concatenate([okt.masks(_parents(r, n), 1) for n, _ in shape])
    q = r.standard_normal((int(starts[-1]), Hq, D)).astype(np.float16)
    most = max(n for n, _ in shape)
    ws = kv.workspace(len(shape), most, max_kv or table.shape[1] * page)
    ws.fill_(0xFF)
    dp, dq = _dev(pages), _dev(q)
    got, lse = _run_attend(kv, dp, table, lens, dq, starts, most, mask, f32=f32, max_kv=max_kv, workspace=ws)
    kv.check()
    for b, (n, L) in enumerate(shape):
        rows = slice(starts[b], starts[b + 1])
        if n:
            _check_rows(got[rows], lse[rows], q[rows], K[b], V[b], okt.visible(mask[rows], L - n, L), D ** -0.5, f32)
    again = _run_attend(kv, dp, table, lens, dq, starts, most, mask, f32=f32, max_kv=max_kv, with_lse=False)[0]
    kv.check()
    np.testing.assert_array_equal(got, again)


@pytest.mark.parametrize("Hq,Hkv,D,n,L", [(4, 2, 128, 3, 500), (8, 2, 64, 40, 200), (2, 2, 256, 20, 90), (8, 1, 128, 64, 3000)])
def test_a_chain_sees_what_the_causal_mask_does(Hq, Hkv, D, n, L):
    """A tree without branches: both calls are within the oracle's bounds, on the same tokens."""
    import torch
    pages, table, K, V = _sequences(5, Hkv, D, 64, [L])
    kv = _cache(Hq, Hkv, D, page_tokens=64, num_pages=pages.shape[0])
    q = _dev(np.random.default_rng(1).standard_normal((n, Hq, D)).astype(np.float16))
    outs = [_full((n, Hq, D), "float32") for _ in range(2)]
    ws = kv.workspace(1, n, L)
    mask = _dev(okt.masks(_parents(None, n, "chain"), 1).view(np.int64))
    for out, tree in zip(outs, (None, mask)):
        kv.attend(_dev(pages), q, _i32([L]), _i32(table), out, q_start=_i32([0, n]), max_q=n, max_kv=L, workspace=ws, tree=tree)
        torch.cuda.synchronize()
    kv.check()
    seen = np.arange(L) <= L - n + np.arange(n)[:, None]
    for out in outs:
        _check_rows(out.cpu().numpy().astype(np.float64), None, q.cpu().numpy(), K[0], V[0], seen, D ** -0.5, True)


@pytest.mark.parametrize("n", [2, 40])
def test_attend_tree_hides_extremes_and_reports(n):
    """Values of the cache's extremes in nodes that a row does not see change nothing, to the bit; a page id outside
    the cache hides its tokens and is reported."""
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    Hq, Hkv, D, page, L = 4, 1, 128, 32, 200
    r = np.random.default_rng(12)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=7)
    x = r.standard_normal((2, 7 * page, 1, D))
    hidden = np.zeros(7 * page, dtype=bool)
    hidden[L - n + 1:L:2] = True  # odd nodes
    outs = []
    for big in (False, True):
        if big:
            x[:, hidden] = np.where(r.random((2, hidden.sum(), 1, D)) < 0.5, 20000, -20000)
        kn, ks, kb, _ = okv.quantise(x[0])
        vn, vs, vb, _ = okv.quantise(x[1])
        pages = okv.pack(kn, ks, kb, vn, vs, vb, page)
        q = _dev(np.random.default_rng(1).standard_normal((n, Hq, D)).astype(np.float16))
        mask = np.full((n, 1), 0x5555555555555555, dtype=np.uint64)
        outs.append(_run_attend(kv, _dev(pages), np.arange(7)[None], [L], q, [0, n], n, mask))
        kv.check()
    np.testing.assert_array_equal(outs[0][0], outs[1][0])
    np.testing.assert_array_equal(outs[0][1], outs[1][1])
    K, V = okv.held(kn, ks, kb), okv.held(vn, vs, vb)
    for bad in (7, -1, 2 ** 31 - 1):
        table = np.arange(7)[None].copy()
        table[0, 1] = bad
        got, lse = _run_attend(kv, _dev(pages), table, [L], q, [0, n], n, mask)
        with pytest.raises(AgemmError, match="page id"):
            kv.check()
        seen = okt.visible(mask, L - n, L)
        seen[:, 32:64] = False
        _check_rows(got, lse, q.cpu().numpy(), K[:L], V[:L], seen, D ** -0.5, True)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- verification

def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _verify_problem(seed, sizes, vocab, drawn, kind="mixed", gap=0.7, sharp=3.0):
    """Trees whose drafts come from q as drafting draws them, node by node without replacement."""
    r = np.random.default_rng(seed)
    T = sum(sizes)
    x = sharp * r.standard_normal((T, vocab))
    y = x + gap * r.standard_normal((T, vocab))
    p, q = _softmax(x), _softmax(y)
    token, parent = np.zeros(T, dtype=np.int64), np.zeros(T, dtype=np.int32)
    starts = _starts(sizes)
    for b, n in enumerate(sizes):
        par = _parents(r, n, kind)
        parent[starts[b]:starts[b + 1]] = par
        for c in range(n):
            kids = [i for i in range(n) if par[i] == c]
            row = starts[b] + c
            z = y[row] + (r.gumbel(size=vocab) if drawn else 0)
            token[[starts[b] + i for i in kids]] = np.argsort(-z)[:len(kids)]
    return dict(T=T, starts=starts, token=token, parent=parent, p=p, q=q if drawn else None,
                u=r.random(T).astype(np.float32))


def _run_verify(kv, c, max_q=None, max_children=1, p=None, q=None, workspace=None, stream=None, **change):
    import torch
    a = {**{k: c[k] for k in ("token", "parent", "starts", "u")}, **change}
    B, T = len(a["starts"]) - 1, len(a["parent"])
    path, count, nxt = _full((T,), "int32"), _full((B,), "int32"), _full((B,), "int64")
    p = _dev(c["p"]) if p is None else p
    q = (None if c["q"] is None else _dev(c["q"])) if q is None else q
    args = [_dev(np.asarray(a["token"], dtype=np.int64)), _i32(a["parent"]), _i32(a["starts"]), _dev(np.asarray(a["u"], dtype=np.float32))]
    torch.cuda.synchronize()
    kv.verify(args[0], args[1], args[2], p, args[3], path, count, nxt, max_q=max_q or int(np.diff(a["starts"]).max()),
              q=q, max_children=max_children, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return path.cpu().numpy(), count.cpu().numpy(), nxt.cpu().numpy()


def _check_verify(got, c, trees=None, least=1e-6, skip=()):
    """Equal to the oracle; no decision of the inputs nearer to its border than `least` (whole rows of binary32
    probabilities count as a sum of 1, which they are to 1e-6 of it: the same on both sides)."""
    path, count, nxt = got
    accepted = 0
    for b in range(len(c["starts"]) - 1):
        if b in skip:
            continue
        rows = slice(c["starts"][b], c["starts"][b + 1])
        n = rows.stop - rows.start
        if n == 0:
            assert count[b] == 0 and nxt[b] == -1
            continue
        want, follow, margin = okt.verify(c["token"][rows], c["parent"][rows], c["p"][rows],
                                          None if c["q"] is None else c["q"][rows], c["u"][rows])
        assert margin > least, (b, margin)
        assert path[rows].tolist() == want + [-1] * (n - len(want)), b
        assert count[b] == len(want) and nxt[b] == follow, (b, nxt[b], follow)
        accepted += len(want) - 1
    return accepted


VERIFIES = [
    # sizes, vocab, drawn, kind, children to expect
    ([1], 1000, True, "chain", 1),
    ([1], 7, False, "chain", 1),
    ([6], 32768, True, "chain", 1),
    ([5, 0, 3, 9, 1], 4099, True, "chain", 1),
    ([5, 0, 3, 9, 1], 4099, False, "chain", 1),
    ([12, 20, 7], 2000, True, "mixed", 20),
    ([12, 20, 7], 2000, True, "mixed", 1),   # more children than said: the last kernel sums them
    ([12, 20, 7], 2001, False, "mixed", 20),
    ([64, 63], 777, True, "star", 64),
    ([65, 130], 512, True, "mixed", 200),
    ([300], 333, False, "mixed", 9),
    ([1024], 65, False, "chain", 1),
    ([25, 25], 65537, True, "mixed", 9),
    ([4] * 40, 131, True, "mixed", 3),
    ([3] * 300, 50, False, "mixed", 2),
    ([3] * 1030, 33, True, "mixed", 2),      # one part a row
    ([2], 200001, True, "chain", 1),
]


@pytest.mark.parametrize("sizes,vocab,drawn,kind,children", VERIFIES)
def test_verify_against_the_oracle(sizes, vocab, drawn, kind, children):
    print(f"[kv verify] {sizes[:5]} {len(sizes)} {vocab} {drawn} {kind} {children}", flush=True)
    kv = _cache(1, 1, 64)
    c = _verify_problem(vocab + len(sizes), sizes, vocab, drawn, kind)
    got = _run_verify(kv, c, max_children=children)
    kv.check()
    # 1030 trees of decisions: the nearest one is nearer
    accepted = _check_verify(got, c, least=1e-6 if len(sizes) < 100 else 1e-8)
    if sum(sizes) > 60 and drawn:
        assert 0 < accepted < sum(sizes) - len(sizes)


@pytest.mark.parametrize("gap", [0.0, 0.2, 5.0])
def test_verify_near_and_far_drafts(gap):
    """Drafts that equal the target (all of a chain accepted), come near it, and miss it (many rejections in a row, so
    more sums than there are rounds)."""
    kv = _cache(1, 1, 64)
    for kind, sizes in (("chain", [9] * 8), ("star", [20] * 8), ("mixed", [30] * 8)):
        c = _verify_problem(int(10 * gap), sizes, 500, True, kind, gap=gap, sharp=1.5)
        got = _run_verify(kv, c, max_children=9)
        kv.check()
        accepted = _check_verify(got, c)
        if gap == 0.0 and kind == "chain":
            assert accepted == 8 * 8


@pytest.mark.parametrize("wait", ["0", "1"])
def test_verify_without_waiting_for_other_workgroups(wait, monkeypatch):
    """Workgroups that give up waiting leave the rest to the last kernel: the same results."""
    monkeypatch.setenv("AGEMM_VERIFY_WAIT_US", wait)
    kv = _cache(1, 1, 64)
    for kind, sizes, vocab in (("star", [20] * 8, 500), ("mixed", [30] * 40, 9000), ("mixed", [12], 70001)):
        c = _verify_problem(7, sizes, vocab, True, kind, gap=2.0, sharp=1.5)
        got = _run_verify(kv, c, max_children=9)
        kv.check()
        _check_verify(got, c)


def test_verify_borders_exactly():
    """Probabilities of few bits and numbers on the borders: a number on a border is not below it, in every part of
    the vocabulary."""
    kv = _cache(1, 1, 64)
    V = 4096 * 3
    p = np.zeros((2, V), dtype=np.float32)
    at = [0, 1023, 1024, 2047, 4095, 4096, 8191, 12287]
    p[:, at] = 1 / 8
    for i, u0 in enumerate(np.arange(8) / 8):
        for d, want in ((0.0, i), (-2.0 ** -24, i - 1), (2.0 ** -24, i)):
            u = max(0.0, u0 + d)
            c = dict(T=1, starts=_starts([1]), token=np.zeros(1), parent=[-1], p=p[:1], q=None, u=[u])
            _, count, nxt = _run_verify(kv, c)
            assert count[0] == 1 and nxt[0] == at[max(0, want)]
    # acceptance: u d(x) < p(x), with d = 1 and with d = 1 / 2
    q = np.zeros((2, V), dtype=np.float32)
    q[:, [0, 5]] = 1 / 2
    for draft, border in ((None, 1 / 8), (q, 1 / 4)):
        for u1, taken in ((border, False), (border - 2.0 ** -24, True), (0.0, True), (0.999, False)):
            c = dict(T=2, starts=_starts([2]), token=[3, 0], parent=[-1, 0], p=p, q=draft, u=[0.0, u1])
            path, count, nxt = _run_verify(kv, c)
            assert count[0] == 1 + taken and path.tolist() == [0, 1 if taken else -1]
            assert nxt[0] == (0 if taken else 1023)
    kv.check()


def test_verify_odd_probabilities_and_numbers():
    """NaN, infinities, negative numbers and numbers past 1; no weight left after a rejection; no weight at all."""
    from shard_decomposed_gemm_amd import AgemmError
    kv = _cache(1, 1, 64)
    V = 3000
    nan, inf = float("nan"), float("inf")
    base = np.zeros((1, V), dtype=np.float32)
    base[0, [7, 2000, 2999]] = 0.25, 0.5, 0.25
    odd = base.copy()
    odd[0, [0, 1, 2, 1500, 2998]] = nan, -1.0, -inf, nan, -0.5
    for p, us in ((base, (0.0, 0.3, 0.9)), (odd, (0.0, 0.3, 0.9))):
        for u, want in zip(us, (7, 2000, 2999)):
            c = dict(T=1, starts=_starts([1]), token=[0], parent=[-1], p=p, q=None, u=[u])
            assert _run_verify(kv, c)[2][0] == want
    for u, want in ((nan, 7), (-3.0, 7), (-inf, 7), (1.0, 2999), (inf, 2999), (5.0, 2999)):
        c = dict(T=1, starts=_starts([1]), token=[0], parent=[-1], p=base, q=None, u=[u])
        assert _run_verify(kv, c)[2][0] == want
    c["p"] = np.full((1, V), inf, dtype=np.float32)  # every entry counts as 1
    c["u"] = [0.5]
    assert _run_verify(kv, c)[2][0] == V // 2
    kv.check()
    # certain drafts that hold all of p, and drafts with q where p has nothing: from p itself
    two = np.repeat(base, 2, 0)
    one = np.zeros((2, V), dtype=np.float32)
    one[:, 9] = 1.0
    for q, token, u1 in ((two, 5, 0.5), (one, 9, 0.0)):
        c = dict(T=2, starts=_starts([2]), token=[0, token], parent=[-1, 0], p=two, q=q, u=[0.3, u1])
        path, count, nxt = _run_verify(kv, c)
        assert count[0] == 1 and nxt[0] == 2000
    kv.check()
    c = dict(T=2, starts=_starts([1, 1]), token=[0, 0], parent=[-1, -1], p=np.concatenate([base, np.full((1, V), nan, np.float32)]),
             q=None, u=[0.5, 0.5])
    path, count, nxt = _run_verify(kv, c)
    assert count.tolist() == [1, 1] and nxt.tolist() == [2000, -1] and path.tolist() == [0, 0]
    with pytest.raises(AgemmError, match="sequence 1: no probability"):
        kv.check()


def test_verify_reports_what_it_cannot_use():
    from shard_decomposed_gemm_amd import AgemmError
    kv = _cache(1, 1, 64)
    c = _verify_problem(5, [6, 6, 6], 400, True)
    c["u"][:] = 0.05  # most drafts are accepted

    def run(match, skip=(), expect=None, **change):
        got = _run_verify(kv, c, max_children=5, **change)
        with pytest.raises(AgemmError, match=match):
            kv.check()
        d = {**c, **{k: np.asarray(v) for k, v in change.items() if k in c}}
        if expect:
            d.update(expect)
        _check_verify(got, d, skip=skip)
        return got

    for bad in (400, -1, 2 ** 62, -2 ** 62):
        token = c["token"].copy()
        token[7] = bad
        run("drafted token", token=token)
    for bad in (5, 100, -2):
        parent = c["parent"].copy()
        parent[8] = bad
        known = parent.copy()
        known[8] = -1
        run("parent", parent=parent, expect=dict(parent=known))
    parent = c["parent"].copy()
    parent[6] = 0  # a root with a parent
    known = parent.copy()
    known[6] = -1
    run("parent", parent=parent, expect=dict(parent=known))
    path, count, nxt = run("query rows", skip=(2,), starts=[0, 6, 12, 19], max_q=7)
    assert count[2] == 0 and nxt[2] == -1 and (path[12:] == PAD).all()
    path, count, nxt = run("query rows", skip=(0, 1, 2), max_q=5)
    assert (count == 0).all() and (nxt == -1).all() and (path == PAD).all()
    got = _run_verify(kv, c, starts=[0, 0, 6, 12], max_children=5)  # rows behind the last sequence
    kv.check()
    assert got[1][0] == 0 and got[2][0] == -1 and (got[0][12:] == PAD).all()


def test_verify_strided_rows_one_row_for_all_and_streams():
    import torch
    kv = _cache(1, 1, 64)
    c = _verify_problem(6, [7, 7], 1003, True)
    first = _run_verify(kv, c, max_children=5)
    _check_verify(first, c)
    wide = [torch.full((14, 1500), float("nan"), device=gu.dev()) for _ in range(2)]
    for w, x in zip(wide, (c["p"], c["q"])):
        w[:, 3:1006] = _dev(x)
    side, ws = torch.cuda.Stream(), kv.verify_workspace(3, 2000)
    for stream, w in ((None, None), (side, ws), (side, None), (None, ws)):
        ws.fill_(0xFF)  # what lies there means nothing
        torch.cuda.synchronize()
        again = _run_verify(kv, c, max_children=5, p=wide[0][:, 3:1006], q=wide[1][:, 3:1006], workspace=w, stream=stream)
        for x, y in zip(first, again):
            np.testing.assert_array_equal(x, y)
    kv.check()
    row = dict(c, p=np.repeat(c["p"][:1], 14, 0), q=np.repeat(c["q"][:1], 14, 0))
    got = _run_verify(kv, row, max_children=5, p=_dev(c["p"][:1]).expand(14, -1), q=_dev(c["q"][:1]).expand(14, -1))
    _check_verify(got, row)


# ---------------------------------------------------------------- commit

COMMITS = [
    # Hkv, D, page, layers, [(nodes, length, path)]
    (2, 128, 32, 1, [(5, 0, [0, 1, 4])]),
    (8, 128, 64, 3, [(13, 777, [0, 2, 3, 9]), (13, 60, [0]), (0, 5, []), (13, 63, [0, 1, 2]), (4, 31, [])]),
    (3, 64, 32, 2, [(40, 20, list(range(1, 40, 2))), (64, 100, [0] + list(range(30, 64)))]),
    (5, 256, 256, 1, [(30, 250, [0, 3, 4, 5, 6, 28, 29])]),
    (1, 128, 128, 66, [(9, 126, [0, 8])]),                                  # layers of two launches
    (2, 64, 64, 1, [(1024, 10, list(range(0, 1024, 2))), (1000, 1, list(range(500, 1000)))]),  # long paths
    (4, 128, 32, 2, [(6, i * 5, [0, 2, 5][:i % 4]) for i in range(70)]),
]


def _commit_problem(seed, Hkv, D, page, layers, shape):
    r = np.random.default_rng(seed)
    width = max(1, max(-(-(n + m) // page) for m, n, _ in shape))
    P = len(shape) * width + 1
    table = r.permutation(P)[:len(shape) * width].reshape(len(shape), width).astype(np.int32)
    before = r.integers(0, 256, (layers, P, Hkv * page * (D + 8)), dtype=np.uint8)
    starts = _starts([m for m, _, _ in shape])
    path = np.full(max(1, starts[-1]), -1, dtype=np.int32)
    for b, (_, _, nodes) in enumerate(shape):
        path[starts[b]:starts[b] + len(nodes)] = nodes
    return dict(table=table, P=P, before=before, starts=starts, path=path[:starts[-1]], lens=[n for _, n, _ in shape],
                count=[len(x) for _, _, x in shape])


def _committed(c, Hkv, D, page, skip=(), lost=()):
    """The pages that come of it."""
    out = []
    for raw in c["before"]:
        parts = list(okv.unpack(raw, Hkv, D, page))
        was = [x.copy() for x in parts]
        for b, n in enumerate(c["lens"]):
            if b in skip:
                continue
            slot = lambda at: int(c["table"][b, at // page]) * page + at % page  # noqa: E731
            for i, x in enumerate(c["path"][c["starts"][b]:c["starts"][b] + c["count"][b]]):
                if (n + i) // page in lost or (n + x) // page in lost:
                    continue
                for now, old in zip(parts, was):
                    now[slot(n + i)] = old[slot(n + x)]
        out.append(okv.pack(*parts, page))
    return out


def _run_commit(kv, c, max_q, stream=None, **change):
    import torch
    a = {**{k: c[k] for k in ("starts", "lens", "path", "count", "table")}, **change}
    pages = [_dev(x) for x in c["before"]]
    new = _full((len(a["lens"]),), "int32")
    args = [_i32(a[k]) for k in ("starts", "lens", "path", "count", "table")]
    torch.cuda.synchronize()
    kv.commit(pages if len(pages) != 1 else pages[0], *args, max_q, new_len=new, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in pages], new.cpu().numpy()


@pytest.mark.parametrize("Hkv,D,page,layers,shape", COMMITS)
def test_commit_moves_the_path_and_nothing_else(Hkv, D, page, layers, shape):
    print(f"[kv commit] {Hkv} {D} {page} {layers} {[s[:2] for s in shape[:4]]}", flush=True)
    c = _commit_problem(D + layers, Hkv, D, page, layers, shape)
    kv = _cache(Hkv, Hkv, D, page_tokens=page, num_pages=c["P"])
    pages, new = _run_commit(kv, c, max(1, max(m for m, _, _ in shape)))
    kv.check()
    for got, want in zip(pages, _committed(c, Hkv, D, page)):
        np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(new, np.array(c["lens"]) + c["count"])


def test_commit_reports_what_it_cannot_use():
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    Hkv, D, page = 2, 64, 32
    shape = [(6, 28, [0, 2, 5]), (8, 30, [0, 1, 7]), (5, 40, [0, 3])]
    c = _commit_problem(9, Hkv, D, page, 2, shape)
    kv = _cache(Hkv, Hkv, D, page_tokens=page, num_pages=c["P"])
    width = c["table"].shape[1]

    def run(match, skip=(), lost=(), max_q=8, **change):
        pages, new = _run_commit(kv, c, max_q, **change)
        with pytest.raises(AgemmError, match=match):
            kv.check()
        kv.check()
        for got, want in zip(pages, _committed(c, Hkv, D, page, skip, lost)):
            np.testing.assert_array_equal(got, want)
        return new.tolist()

    for bad in ([0, 0, 7], [0, 7, 1], [-1, 1, 7], [0, 1, 8], [2 ** 31 - 1, 1, 2], [0, 1, -2 ** 31]):
        path = c["path"].copy()
        path[6:9] = bad
        assert run("path", (1,), path=path) == [31, 30, 42]
    for bad in (9, -1, 2 ** 31 - 1, -2 ** 31):
        assert run("path", (1,), count=[3, bad, 2]) == [31, 30, 42]
    for bad in (-1, 2 ** 31 - 1, -2 ** 31, 32 * width - 7):
        assert run("length", (1,), lens=[28, bad, 40]) == [31, bad, 42]
    assert run("query rows", (1,), max_q=7) == [31, 30, 42]
    assert run("query rows", (2,), starts=[0, 6, 14, 20]) == [31, 33, 40]
    assert run("query rows", (0,), starts=[-1, 6, 14, 19]) == [28, 33, 42]
    # a page that is not there: nodes on it or bound for it stay, the others move
    for bad in (c["P"], -1, 2 ** 31 - 1):
        t = c["table"].copy()
        t[0, 1] = bad
        d = dict(c, lens=c["lens"][:1], count=c["count"][:1], starts=c["starts"][:2], path=c["path"][:6], table=c["table"][:1])
        pages, new = _run_commit(kv, d, 8, table=t[:1])
        with pytest.raises(AgemmError, match="page id"):
            kv.check()
        for got, want in zip(pages, _committed(d, Hkv, D, page, lost=(1,))):
            np.testing.assert_array_equal(got, want)
        assert new.tolist() == [31]
    # lengths alone, no layers
    new = _full((3,), "int32")
    kv.commit([], _i32(c["starts"]), _i32(c["lens"]), _i32(c["path"]), _i32(c["count"]), _i32(c["table"]), 8, new_len=new)
    torch.cuda.synchronize()
    kv.check()
    assert new.tolist() == [31, 33, 42]


# ---------------------------------------------------------------- together

def _step_tensors(kv, B, N, T, Hq, D, V, layers):
    import torch
    e = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=gu.dev())  # noqa: E731
    return dict(mask=e(T, 1, dtype=torch.int64), pos=e(T, dtype=torch.int64), slots=e(T, dtype=torch.int64),
                total=e(B, dtype=torch.int32), qr=e(T, Hq, D, dtype=torch.float16),
                out=[e(T, Hq, D, dtype=torch.float16) for _ in range(layers)], path=e(T, dtype=torch.int32),
                count=e(B, dtype=torch.int32), next=e(B, dtype=torch.int64), new=e(B, dtype=torch.int32))


def test_speculative_steps_in_a_graph_and_eager():
    """A step - layout, append, attention over the tree, verification, commit - captured once and replayed with new
    drafts and with the lengths that the step before it left; every replay equals the eager calls, and every accepted
    token's attention what a cache filled token by token gives."""
    import torch
    Hq, Hkv, D, page, V, layers, B, N = 8, 2, 128, 32, 501, 2, 3, 10
    T = B * N + 2  # two rows of padding
    r = np.random.default_rng(2)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=B * 6)
    table = _i32(r.permutation(B * 6).reshape(B, 6))
    rope = _dev(np.concatenate([f(np.arange(192)[:, None] * 10000.0 ** (-2 * np.arange(D // 2) / D)) for f in (np.cos, np.sin)],
                               1).astype(np.float32))
    pages = [kv.new_pages() for _ in range(layers)]
    sizes = [N, N - 3, N]
    starts = _i32(_starts(sizes))
    x = [torch.zeros(T, Hq + 2 * Hkv, D, dtype=torch.float16, device=gu.dev()) for _ in range(layers)]
    parent, token = _full((T,), "int32", -1), torch.zeros(T, dtype=torch.int64, device=gu.dev())
    p, q = (torch.full((T, V), 1 / V, device=gu.dev()) for _ in range(2))
    u, lens = torch.zeros(T, device=gu.dev()), torch.zeros(B, dtype=torch.int32, device=gu.dev())
    ws, vws = kv.workspace(B, N, 192), kv.verify_workspace(B, V)

    def step(pages, t, ws, vws):
        kv.tree(parent, starts, lens, table, N, t["mask"], positions=t["pos"], slots=t["slots"], total_len=t["total"])
        for i in range(layers):
            kv.append(pages[i], q=x[i][:, :Hq], k=x[i][:, Hq:Hq + Hkv], v=x[i][:, Hq + Hkv:], slots=t["slots"],
                      positions=t["pos"], rope=rope, q_out=t["qr"])
            kv.attend(pages[i], t["qr"], t["total"], table, t["out"][i], q_start=starts, max_q=N, max_kv=192, workspace=ws,
                      tree=t["mask"])
        kv.verify(token, parent, starts, p, u, t["path"], t["count"], t["next"], max_q=N, q=q, max_children=N, workspace=vws)
        kv.commit(pages, starts, lens, t["path"], t["count"], table, N, new_len=t["new"])

    t, e = (_step_tensors(kv, B, N, T, Hq, D, V, layers) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step([y.clone() for y in pages], t, ws, vws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pages, t, ws, vws)
    eager = [y.clone() for y in pages]
    plain = [y.clone() for y in pages]
    lens.copy_(torch.tensor([0, 5, 30]))
    for i in range(layers):  # what was there before
        y = torch.randn(35, Hkv, D, device=gu.dev()).half()
        at = torch.tensor([(1, a) for a in range(5)] + [(2, a) for a in range(30)], device=gu.dev())
        slots = table.long()[at[:, 0], at[:, 1] // page] * page + at[:, 1] % page
        for z in (pages[i], eager[i], plain[i]):
            kv.append(z, k=y, v=y, slots=slots)
    for turn in range(5):
        c = _verify_problem(turn, sizes, V, True, gap=0.3)
        n = c["T"]
        parent[:n], token[:n] = _dev(c["parent"]), _dev(c["token"])
        p[:n], q[:n], u[:n] = _dev(c["p"]), _dev(c["q"]), _dev(c["u"])
        for y in x:
            y.copy_(torch.randn(y.shape, device=gu.dev()))
        for z in (t, e):
            z["path"].fill_(PAD)
            for o in z["out"]:
                o.fill_(PAD)
        ws.fill_(0xFF)
        vws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        step(eager, e, None, None)
        torch.cuda.synchronize()
        kv.check()
        for k in t:
            for a, b in zip(t[k], e[k]) if k == "out" else ((t[k], e[k]),):
                assert torch.equal(a, b), k
        for a, b in zip(pages, eager):
            assert torch.equal(a, b)
        _check_verify([t[k].cpu().numpy() for k in ("path", "count", "next")], c)
        # the accepted tokens one after another, as a decoder without drafts appends and attends
        path, count, start, old = t["path"].tolist(), t["count"].tolist(), starts.tolist(), lens.tolist()
        for b in range(B):
            for i in range(count[b]):
                row = start[b] + path[start[b] + i]
                at = old[b] + i
                slot = table[b, at // page].long()[None] * page + at % page
                for j in range(layers):
                    xr = x[j][row:row + 1]
                    qr = torch.zeros(1, Hq, D, dtype=torch.float16, device=gu.dev())
                    kv.append(plain[j], q=xr[:, :Hq], k=xr[:, Hq:Hq + Hkv], v=xr[:, Hq + Hkv:], slots=slot,
                              positions=torch.tensor([at], device=gu.dev()), rope=rope, q_out=qr)
                    one = _full((1, Hq, D), "float32")
                    kv.attend(plain[j], qr, _i32([at + 1]), table[b:b + 1], one)
                    # both within the rounding of weights and output of the value (see _check_rows), |V| below 8
                    assert (one - t["out"][j][row:row + 1].float()).abs().max().item() <= 2 * 8 * 2.0 ** -11
        for b in range(B):
            slots = torch.tensor([int(table[b, a // page]) * page + a % page for a in range(old[b] + count[b])], device=gu.dev())
            for j in range(layers):
                kept = [torch.zeros(2, len(slots), Hkv, D, dtype=torch.float16, device=gu.dev()) for _ in range(2)]
                kv.read(pages[j], slots, kept[0][0], kept[0][1])
                kv.read(plain[j], slots, kept[1][0], kept[1][1])
                assert torch.equal(*kept)
        lens.copy_(t["new"])
    assert lens.tolist() != [5, 10, 35]  # some drafts were accepted on the way


def test_calls_at_once_on_streams():
    """Two verifications whose workgroups wait for each other, two attention calls with trees, a layout and a commit in
    flight together, each with a workspace of its own."""
    import torch
    Hq, Hkv, D, page, n = 8, 2, 128, 32, 20
    pages, table, K, V = _sequences(22, Hkv, D, page, [3000, 900])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    r = np.random.default_rng(5)
    dp, dt, lens, starts = _dev(pages), _i32(table), _i32([3000, 900]), _i32([0, n, 2 * n])
    masks = [np.concatenate([okt.masks(_parents(r, n), 1) for _ in range(2)]) for _ in range(2)]
    dm = [_dev(x.view(np.int64)) for x in masks]
    qs = [r.standard_normal((2 * n, Hq, D)).astype(np.float16) for _ in range(2)]
    dq = [_dev(x) for x in qs]
    outs = [_full((2 * n, Hq, D), "float32") for _ in range(2)]
    ws = [kv.workspace(2, n, 4096) for _ in range(2)]
    problems = [_verify_problem(30 + i, [30] * 12, 20011, True, "mixed", gap=1.5) for i in range(2)]
    dev = [{k: _dev(x[k]) for k in ("token", "p", "q", "u")} | dict(parent=_i32(x["parent"]), starts=_i32(x["starts"])) for x in problems]
    got = [(_full((360,), "int32"), _full((12,), "int32"), _full((12,), "int64")) for _ in range(2)]
    vws = [kv.verify_workspace(12, 20011) for _ in range(2)]
    parent, mask = _i32(_parents(r, n) * 2), _full((2 * n, 1), "int64")
    c = _commit_problem(3, Hkv, D, page, 1, [(13, 60, [0, 2, 3, 9])])
    other, old = _cache(Hkv, Hkv, D, page_tokens=page, num_pages=c["P"]), _dev(c["before"][0])
    args = [_i32(c[k]) for k in ("starts", "lens", "path", "count", "table")]
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    for turn in range(10):
        for i in (0, 1):
            d = dev[i]
            kv.verify(d["token"], d["parent"], d["starts"], d["p"], d["u"], *got[i], max_q=30, q=d["q"], max_children=9,
                      workspace=vws[i], stream=streams[i])
            kv.attend(dp, dq[i], lens, dt, outs[i], q_start=starts, max_q=n, workspace=ws[i], stream=streams[2 + i], tree=dm[i])
        kv.tree(parent, starts, lens, None, n, mask, stream=streams[4])
        if turn == 0:
            other.commit(old, *args, 13, stream=streams[5])
    torch.cuda.synchronize()
    kv.check()
    other.check()
    for i in (0, 1):
        _check_verify([x.cpu().numpy() for x in got[i]], problems[i])
        for b, L in enumerate((3000, 900)):
            rows = slice(b * n, (b + 1) * n)
            _check_rows(outs[i][rows].cpu().numpy().astype(np.float64), None, qs[i][rows], K[b], V[b],
                        okt.visible(masks[i][rows], L - n, L), D ** -0.5, True)
    np.testing.assert_array_equal(old.cpu().numpy(), _committed(c, Hkv, D, page)[0])


def test_two_graphs_share_workspaces():
    """Attention and verification captured into two graphs with the same workspaces, replayed in turn with eager calls in
    between: what one leaves there does not matter to the other."""
    import torch
    Hq, Hkv, D, page = 8, 1, 64, 32
    sides = []
    ws = vws = None
    for lens, n, vocab in (([4000, 70], 33, 5003), ([2500, 2600, 900], 9, 777)):
        B = len(lens)
        pages, table, _, _ = _sequences(B, Hkv, D, page, lens)
        kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
        if ws is None:
            ws, vws = kv.workspace(3, 33, 4096), kv.verify_workspace(3, 5003)
        r = np.random.default_rng(B)
        t = dict(dp=_dev(pages), dt=_i32(table), lens=_i32(lens), starts=_i32(_starts([n] * B)),
                 q=_dev(r.standard_normal((B * n, Hq, D)).astype(np.float16)), out=_full((B * n, Hq, D), "float32"),
                 mask=_dev(np.concatenate([okt.masks(_parents(r, n), 1) for _ in lens]).view(np.int64)))
        c = _verify_problem(B, [n] * B, vocab, True, gap=1.0)
        d = {k: _dev(c[k]) for k in ("token", "p", "q", "u")}
        t.update(d, parent=_i32(c["parent"]), path=_full((B * n,), "int32"), count=_full((B,), "int32"), next=_full((B,), "int64"))

        def step(kv=kv, t=t, n=n):
            kv.attend(t["dp"], t["q"], t["lens"], t["dt"], t["out"], q_start=t["starts"], max_q=n, workspace=ws, tree=t["mask"])
            kv.verify(t["token"], t["parent"], t["starts"], t["p"], t["u"], t["path"], t["count"], t["next"], max_q=n, q=t["q_"],
                      max_children=9, workspace=vws)
        t["q_"], t["q"] = t["q"], _dev(r.standard_normal((B * n, Hq, D)).astype(np.float16))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        step()
        torch.cuda.synchronize()
        _check_verify([t[k].cpu().numpy() for k in ("path", "count", "next")], c)
        sides.append((kv, t, graph, {k: t[k].clone() for k in ("out", "path", "count", "next")}, step))
    for turn in range(4):
        for kv, t, graph, want, step in sides:
            for k in want:
                t[k].fill_(PAD)
            graph.replay()
            torch.cuda.synchronize()
            for k, x in want.items():
                assert torch.equal(t[k], x), k
            if turn % 2:
                step()
            torch.cuda.synchronize()
            kv.check()


def test_tree_partials_of_ranks_combine():
    """Flash Decode with a tree: ranks that hold parts of the cached tokens attend without a mask, the last one with the
    tree; the combine of their partials is the attention over all."""
    import torch
    from shard_decomposed_gemm_amd import FdCombine
    W, Hq, Hkv, D, page, n = 2, 8, 2, 128, 32, 6
    r = np.random.default_rng(3)
    pages, table, K, V = _sequences(8, Hkv, D, page, [100, 40 + n])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = r.standard_normal((n, Hq, D)).astype(np.float16)
    mask = okt.masks(_parents(r, n), 1)
    dp, dq = _dev(pages), _dev(q)
    o = [_full((n, Hq, D), "float32") for _ in range(W)]
    lse = [_full((n, Hq), "float32") for _ in range(W)]
    kv.attend(dp, dq, _i32([100]), _i32(table[:1]), o[0], lse=lse[0], q_start=_i32([0, n]), max_q=n, causal=False)
    kv.attend(dp, dq, _i32([40 + n]), _i32(table[1:]), o[1], lse=lse[1], q_start=_i32([0, n]), max_q=n, tree=_dev(mask.view(np.int64)))
    torch.cuda.synchronize()
    kv.check()
    fdc = FdCombine(W, n * Hq, D, heads_per_tile=8, out_dtype="f32")
    O = _full((n * Hq, D), "float32")
    sp, sc = fdc.streams()
    torch.cuda.synchronize()
    fdc.produce([x.view(n * Hq, D) for x in o], [x.view(n * Hq) for x in lse], stream=sp)
    fdc.run_fused(O, stream=sc)
    torch.cuda.synchronize()
    fdc.check()
    fdc.close()
    seen = np.concatenate([np.ones((n, 100), dtype=bool), okt.visible(mask, 40, 40 + n)], 1)
    # the combine adds two weights and products to what _check_rows allows: within its 64 * 2^-24
    _check_rows(O.cpu().numpy().astype(np.float64).reshape(n, Hq, D), None, q, np.concatenate(K), np.concatenate(V), seen,
                D ** -0.5, True)


def test_binding_refuses_wrong_tensors():
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    kv = _cache(2, 1, 64, page_tokens=32, num_pages=4)
    pages = kv.new_pages()
    parent, starts, lens, table = _i32([-1, 0, 0]), _i32([0, 3]), _i32([5]), _i32([[0, 1]])
    mask, slots = _full((3, 1), "int64", 0), _full((3,), "int64", 0)
    token, u, p = slots.clone(), torch.zeros(3, device=gu.dev()), torch.ones(3, 10, device=gu.dev())
    path, count, nxt = _i32([0, -1, -1]), _i32([1]), _full((1,), "int64", 0)
    q, out = torch.zeros(3, 2, 64, dtype=torch.float16, device=gu.dev()), torch.zeros(3, 2, 64, device=gu.dev())
    for err, call in [
        (TypeError, lambda: kv.tree(parent.long(), starts, lens, table, 3, mask)),
        (ValueError, lambda: kv.tree(parent, starts[:1], lens, table, 3, mask)),
        (TypeError, lambda: kv.tree(parent, starts, lens, table, 3, mask.int())),
        (ValueError, lambda: kv.tree(parent, starts, lens, table, 3, mask[:2])),
        (ValueError, lambda: kv.tree(parent, starts, lens, table[:0], 3, mask)),
        (AgemmError, lambda: kv.tree(parent, starts, lens, table, 65, mask)),
        (AgemmError, lambda: kv.tree(parent, starts, lens, None, 3, mask, slots=slots)),
        (AgemmError, lambda: kv.tree(parent, starts, lens, table, 3, mask, total_len=lens)),
        (ValueError, lambda: kv.attend(pages, q, lens, table, out, q_start=starts, max_q=3, tree=mask[:2])),
        (TypeError, lambda: kv.attend(pages, q, lens, table, out, q_start=starts, max_q=3, tree=mask.int())),
        (AgemmError, lambda: kv.attend(pages, q, lens, table, out, q_start=starts, max_q=3, tree=mask, causal=False)),
        (AgemmError, lambda: kv.attend(pages, q, lens, table, out, q_start=starts, max_q=3, tree=mask.expand(3, 17).contiguous())),
        (TypeError, lambda: kv.verify(token, parent, starts, p.half(), u, path, count, nxt, 3)),
        (ValueError, lambda: kv.verify(token, parent, starts, p[:2], u, path, count, nxt, 3)),
        (ValueError, lambda: kv.verify(token, parent, starts, p, u, path, count, nxt, 3, q=p[:, :9])),
        (ValueError, lambda: kv.verify(token, parent, starts, p.t().contiguous().t(), u, path, count, nxt, 3)),
        (TypeError, lambda: kv.verify(token.int(), parent, starts, p, u, path, count, nxt, 3)),
        (TypeError, lambda: kv.verify(token, parent, starts, p, u.double(), path, count, nxt, 3)),
        (AgemmError, lambda: kv.verify(token, parent, starts, p, u, path, count, nxt, 3, workspace=_full((16,), "uint8")[:4])),
        (TypeError, lambda: kv.verify(token, parent, starts, p, u, path, count, nxt, 3, workspace=u)),
        (AgemmError, lambda: kv.verify(token, parent, starts, p, u, path, count, nxt, 1025)),
        (AgemmError, lambda: kv.verify(token, parent, starts, p, u, path, count, nxt, 3, max_children=0)),
        (TypeError, lambda: kv.commit(pages.int(), starts, lens, path, count, table, 3)),
        (ValueError, lambda: kv.commit([pages, pages[:2]], starts, lens, path, count, table, 3)),
        (AgemmError, lambda: kv.commit([pages, pages], starts, lens, path, count, table, 3)),
        (TypeError, lambda: kv.commit(pages, starts, lens, path.long(), count, table, 3)),
        (AgemmError, lambda: kv.commit(pages, starts, lens, path, count, table, 3, new_len=lens)),
    ]:
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()
    kv.check()
