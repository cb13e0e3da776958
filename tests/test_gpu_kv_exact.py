"""GPU tests of attention over the 4-bit cache on inputs whose outputs are exact (tests/kv_exact.py), so that a block
left out, taken twice or paired with another block's values shows at any length."""
import numpy as np
import pytest

from tests import gpu_util as gu
from tests import kv_exact as kx

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
