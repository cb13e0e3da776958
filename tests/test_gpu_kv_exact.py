"""GPU tests of attention over the 4-bit cache on inputs whose outputs are exact (tests/kv_exact.py), so that a block
left out, taken twice or paired with another block's values shows at any length."""
import numpy as np
import pytest

from tests import gpu_util as gu
from tests import kv_exact as kx
from tests.test_gpu_kv import BATCHES, LONG

pytestmark = pytest.mark.gpu


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(gu.dev())


def _attend(kv, pages, table, lens, starts, max_q, f32, q_off=None, max_kv=None):
    """Outputs (T, Hq, D) and lse (T, Hq) of queries of -1."""
    import torch
    T = int(starts[-1])
    q = torch.full((T, kv.Hq, kv.D), -1.0, dtype=torch.float16, device=gu.dev())
    out = torch.full((T, kv.Hq, kv.D), 9.0, dtype=torch.float32 if f32 else torch.float16, device=gu.dev())
    lse = torch.full((T, kv.Hq), 9.0, dtype=torch.float32, device=gu.dev())
    i32 = lambda x: None if x is None else _dev(np.asarray(x, dtype=np.int32))  # noqa: E731
    kv.attend(pages, q, i32(lens), table, out, lse=lse, q_start=i32(starts), max_q=max_q, q_off=i32(q_off),
              scale=kx.SCALE, max_kv=max_kv)
    torch.cuda.synchronize()
    kv.check()
    return out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------- the longest sequences

@pytest.mark.parametrize("queries,lens", [
    (1, [(1 << 31) - 1]), (1, [(1 << 31) - 31]), (1, [300, (1 << 31) - 1, 5000]), (33, [(1 << 31) - 1])])
def test_attend_lengths_up_to_the_largest_int32(queries, lens):
    """Sequences of up to 2^31 - 1 tokens, all on the same four pages over and over."""
    import torch
    from shard_decomposed_gemm_amd import KvCache
    print(f"[kv longest] {queries} {lens}", flush=True)
    D, page, P = 64, 256, 4
    kn, vn, shown = kx.tokens(np.random.default_rng(len(lens)), (P * page, 1), D, top=1)
    kn[0], shown[0] = 0, True
    kv = KvCache(1, 1, D, page_tokens=page, num_pages=P)
    table = (torch.arange(1 << 23, device=gu.dev(), dtype=torch.int32) % P).expand(len(lens), -1)
    starts = np.arange(len(lens) + 1) * queries
    got, lse = _attend(kv, _dev(kx.pack(kn, vn, page)), table, lens, starts, queries, True)
    count, total = np.cumsum(shown[:, 0].astype(np.int64)), np.cumsum((shown * vn[:, 0]).astype(np.int64), 0)
    for i, L in enumerate(lens):
        for row in range(queries):
            whole, rest = divmod(L - queries + 1 + row, P * page)
            n = whole * count[-1] + (count[rest - 1] if rest else 0)
            O = (whole * total[-1] + (total[rest - 1] if rest else 0)) / n
            # a run's sums stay below 2^24 tokens; the waves and the at most 256 runs add up with a rounding each
            assert kx.close(got[i * queries + row], lse[i * queries + row], O[None], np.array([n]), True,
                            (8 + 256) * kx.ROUND).all(), (i, row)


# ---------------------------------------------------------------- nothing to do

@pytest.mark.parametrize("max_q", [1, 50])
def test_attend_an_empty_batch_with_long_lengths(max_q):
    import torch
    from shard_decomposed_gemm_amd import KvCache
    kv = KvCache(8, 2, 64, page_tokens=64, num_pages=2)
    none = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device=gu.dev())  # noqa: E731
    assert kv.workspace(0, max_q, 262144).numel() > 0
    kv.attend(kv.new_pages(), none(0, 8, 64, dtype=torch.float16), none(0), none(0, 5000), none(0, 8, 64, dtype=torch.float32),
              q_start=none(1), max_q=max_q)
    torch.cuda.synchronize()
    kv.check()


# ---------------------------------------------------------------- one workspace for a server's calls

def test_one_workspace_for_every_smaller_call():
    """The workspace of the largest batch, chunk and length takes smaller calls, which split their work further."""
    import torch
    from shard_decomposed_gemm_amd import KvCache
    Hq, Hkv, D, page, P = 16, 2, 64, 64, 40
    r = np.random.default_rng(1)
    kn, vn, shown = kx.tokens(r, (P * page, Hkv), D)
    kn[0], shown[0] = 0, True
    kv = KvCache(Hq, Hkv, D, page_tokens=page, num_pages=P)
    pages, L = _dev(kx.pack(kn, vn, page)), P * page
    ws = kv.workspace(600, 300, 2 * L)
    count, total = np.cumsum(shown, 0), np.cumsum(shown[..., None] * vn.astype(np.int64), 0)
    for batch, nq, max_kv in ((600, 1, L), (300, 1, L), (3, 1, L), (1, 1, 2 * L), (200, 3, L), (1, 4, L), (1, 40, L), (2, 300, L)):
        T = batch * nq
        q = torch.full((T, Hq, D), -1.0, dtype=torch.float16, device=gu.dev())
        out, lse = torch.full((T, Hq, D), 9.0, device=gu.dev()), torch.full((T, Hq), 9.0, device=gu.dev())
        kv.attend(pages, q, torch.full((batch,), L, dtype=torch.int32, device=gu.dev()),
                  torch.arange(P, dtype=torch.int32, device=gu.dev()).expand(batch, P), out, lse=lse, max_q=nq,
                  q_start=torch.arange(batch + 1, dtype=torch.int32, device=gu.dev()) * nq, scale=kx.SCALE, max_kv=max_kv,
                  workspace=ws)
        torch.cuda.synchronize()
        kv.check()
        last = L - nq + np.arange(T) % nq
        n = np.repeat(count[last], Hq // Hkv, 1)
        O = np.repeat(total[last], Hq // Hkv, 1) / n[..., None]
        assert kx.close(out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), O, n, True).all()


# ---------------------------------------------------------------- tiny weights

@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("part", [3326.99, 1663.5, 52.9, 3.98])
def test_attend_a_flat_tail_under_one_large_weight(part, queries, f32):
    """One token has all but a little of the weight, and 2^18 others the same tiny weight each, part x 2^-36 of the
    largest: a multiple of binary16's least number that the cut to two numbers (the rounding to one) makes whole."""
    import torch
    from shard_decomposed_gemm_amd import KvCache
    D, page, L = 64, 256, 1 << 18
    P = L // page
    kn, vn = np.zeros((L, 1, D), dtype=np.uint8), np.full((L, 1, D), 15, dtype=np.uint8)
    kn[:, :, 0], kn[0], vn[0] = 15, 0, 0
    kv = KvCache(1, 1, D, page_tokens=page, num_pages=P)
    q = torch.zeros(queries, 1, D, dtype=torch.float16, device=gu.dev())
    q[..., 0] = -1
    out = torch.empty(queries, 1, D, dtype=torch.float32 if f32 else torch.float16, device=gu.dev())
    lse = torch.empty(queries, 1, device=gu.dev())
    scale = float(np.float32((36 - np.log2(part)) * np.log(2) / 15))
    i32 = lambda x: _dev(np.asarray(x, dtype=np.int32))  # noqa: E731
    kv.attend(_dev(kx.pack(kn, vn, page)), q, i32([L]), i32(np.arange(P)[None]), out, lse=lse, q_start=i32([0, queries]),
              max_q=queries, causal=False, scale=scale)
    torch.cuda.synchronize()
    kv.check()
    w = np.exp(-15 * scale)
    total = 1 + (L - 1) * w
    want = 15 * (L - 1) * w / total
    # The score -15 scale is one exact product; its factor scale log2(e) and the exponent round three times, and the
    # power once more: d of a weight. 256 runs; a wave of few rows adds 32 times in a lane of its four blocks, one of
    # many rows 512 (and both up to 128 products in a row), then the waves and runs add up.
    d = 3 * 15 * scale * kx.ROUND + 2.0 ** -22
    sums = (512 + 128 + 8 + 256) * kx.ROUND
    bound = want * (2 * d + 2 * sums + (2.0 ** -21 if f32 else 2.0 ** -11)) + 15 * L * (2.0 ** -36 if f32 else 2.0 ** -37)
    bound += want * 2.0 ** -23 if f32 else max(want * 2.0 ** -11, 2.0 ** -25)
    assert (np.abs(out.cpu().numpy().astype(np.float64) - want) <= bound).all()
    got = lse.cpu().numpy().astype(np.float64)
    assert (np.abs(got - np.log(total)) <= (total - 1) / total * (d + sums) + sums + 2.0 ** -18).all()


# ---------------------------------------------------------------- every token once

BIG = [
    # Hq, Hkv, D, page, [(queries, length)], q_off, max_kv: single tokens of long sequences, prompts on long ones
    (12, 1, 128, 256, [(1, 262144)], None, None),
    (3, 3, 64, 32, [(1, 131072 + 77)], None, None),
    (4, 2, 256, 64, [(1, 50001), (1, 9), (1, 20000)], None, None),
    (8, 2, 128, 64, [(1, 4000 + 131 * i) for i in range(40)], None, None),
    (8, 1, 64, 64, [(5, 60000)], None, None),
    (1, 1, 128, 64, [(1000, 5000)], None, None),
    (16, 2, 128, 64, [(96, 20000), (200, 7777)], None, None),
    (6, 1, 256, 128, [(60, 9000)], None, None),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,shape,q_off,max_kv", LONG + BATCHES + BIG)
def test_attend_takes_every_token_once(Hq, Hkv, D, page, shape, q_off, max_kv, f32):
    """Runs, tiles and their joins leave out no block, take none twice, and pair keys with their own values."""
    from shard_decomposed_gemm_amd import KvCache
    print(f"[kv every] {Hq} {Hkv} {D} {page} {shape[:4]} {len(shape)} {q_off} {max_kv} {f32}", flush=True)
    lens = [n for _, n in shape]
    starts = np.concatenate([[0], np.cumsum([q for q, _ in shape])])
    c = kx.Sequences(Hq + D, Hkv, D, page, lens)
    kv = KvCache(Hq, Hkv, D, page_tokens=page, num_pages=c.pages.shape[0])
    got, lse = _attend(kv, _dev(c.pages), _dev(c.table), lens, starts, max(n for n, _ in shape), f32, q_off, max_kv)
    for i, (n, L) in enumerate(shape):
        off = L - n if q_off is None else q_off[i]
        O, count = c.rows(i, np.clip(off + np.arange(n) + 1, 0, L), Hq // Hkv)
        rows = slice(starts[i], starts[i + 1])
        assert kx.close(got[rows], lse[rows], O, count, f32).all(), i


# ---------------------------------------------------------------- far scores

@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_attend_scores_of_any_size(sign, queries, f32):
    """Shown tokens share one score, the largest, of 2^14 to 2^120: where binary32 has no fractions left of it too, they
    have equal weights and the hidden ones none."""
    import torch
    from shard_decomposed_gemm_amd import KvCache
    D, page, L = 64, 64, 3200
    r = np.random.default_rng(sign + 1)
    kn, vn, shown = kx.tokens(r, (L, 1), D)
    level = 15 if sign > 0 else 7
    kn = np.maximum(kn, level) if sign < 0 else np.minimum(kn, 15)
    at = r.integers(0, D, (L, 1, 1))
    np.put_along_axis(kn, at, np.full((L, 1, 1), 15 if sign < 0 else 7, dtype=np.uint8), -1)  # 8 or more off the level
    kn[0], shown[0] = level, True
    kn[shown] = level
    kv = KvCache(2, 1, D, page_tokens=page, num_pages=L // page)
    pages, table = _dev(kx.pack(kn, vn, page)), _dev(np.arange(L // page, dtype=np.int32)[None])
    q = torch.full((queries, 2, D), float(sign), dtype=torch.float16, device=gu.dev())
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=gu.dev())  # noqa: E731
    last = np.arange(L - queries, L)
    n = np.cumsum(shown[:, 0])[last]
    O = np.cumsum(shown * vn[:, 0].astype(np.int64), 0)[last] / n[:, None]
    for k in (4, 8, 13, 14, 15, 16, 17, 18, 19, 20, 21, 22, 24, 27, 33, 50, 90, 110):
        for scale in (2.0 ** k, 1.37 * 2.0 ** k):
            scale = float(np.float32(scale))
            out = torch.empty(queries, 2, D, dtype=torch.float32 if f32 else torch.float16, device=gu.dev())
            lse = torch.empty(queries, 2, device=gu.dev())
            kv.attend(pages, q, i32(L), table, out, lse=lse, q_start=i32(0, queries), max_q=queries, scale=scale)
            torch.cuda.synchronize()
            kv.check()
            got = out.cpu().numpy().astype(np.float64)
            # equal weights, a power of two or that of a fraction that all share, cut or rounded alike: means, off by
            # the weight's rounding, the sums' (1600 numbers in a row at most) and the output's
            bound = O * ((2.0 ** -21 if f32 else 2.0 ** -11) + 3200 * kx.ROUND)
            bound = bound + (O * 2.0 ** -23 if f32 else np.maximum(O * 2.0 ** -11, 2.0 ** -25))
            assert (np.abs(got - O[:, None]) <= bound[:, None]).all(), (k, scale)
            want = sign * level * D * scale + np.log(n)
            # the factor, the product, the logarithm's sum and the product with ln 2
            assert (np.abs(lse.cpu().numpy() - want[:, None]) <= np.abs(want[:, None]) * 5 * kx.ROUND + 2.0 ** -13).all(), (k, scale)
