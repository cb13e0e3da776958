"""GPU attention with a tree in the forms that tests/test_gpu_kv_tree.py does not reach (tests/test_kv_tree_bounds.py counts them)."""
import numpy as np
import pytest

from oracle import kvtree as okt
from tests import test_gpu_kv_tree as tree
from tests.test_gpu_kv import _cache, _dev, _sequences

pytestmark = pytest.mark.gpu

FORMS = [
    # Hq, Hkv, D, page, [(queries, length)], max_kv: tiles of 128 rows of D 128 in several runs, and every tile's runs
    # joined by a workgroup a row and by waves
    (40, 8, 128, 64, tree._batch(15, 13, 2338), 2338),
    (40, 8, 128, 64, tree._batch(20, 13, 2305), 2305),
    (32, 8, 128, 64, tree._batch(16, 19, 5523), 5523),
    (16, 1, 128, 32, [(9, 2036)], 2036),
    (1, 1, 128, 32, [(1, 1730)], 1730),
    (1, 1, 128, 64, [(34, 1772)], 1772),
    (1, 1, 256, 64, [(1, 1955)], 1955),
    (24, 2, 64, 64, [(15, 8865)], 8865),
    (1, 1, 64, 32, [(33, 1996)], 1996),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,shape,max_kv", FORMS)
def test_attend_a_tree_in_the_other_forms(Hq, Hkv, D, page, shape, max_kv, f32):
    tree.test_attend_a_tree_in_every_form(Hq, Hkv, D, page, shape, max_kv, f32)


@pytest.mark.parametrize("q_off", [False, True])
@pytest.mark.parametrize("scale", [0.09, 0.0, -0.2])
def test_single_queries_without_starts(q_off, scale):
    """One node a sequence and no q_start, rows behind the last sequence; scores of either sign."""
    import torch
    Hq, Hkv, D, page, lens = 8, 2, 128, 32, [1, 40, 333, 0, 2500]
    r = np.random.default_rng(4)
    B = len(lens)
    pages, table, K, V = _sequences(3, Hkv, D, page, lens)
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = r.standard_normal((B + 2, Hq, D)).astype(np.float16)
    mask = r.integers(0, 2 ** 63, (B + 2, 1), dtype=np.uint64) if q_off else np.full((B + 2, 1), 1, dtype=np.uint64)
    offs = [max(0, n - 50) for n in lens] if q_off else [n - 1 for n in lens]
    out, lse = tree._full((B + 2, Hq, D), "float32"), tree._full((B + 2, Hq), "float32")
    kv.attend(_dev(pages), _dev(q), tree._i32(lens), tree._i32(table), out, lse=lse, q_off=tree._i32(offs) if q_off else None,
              scale=scale, tree=_dev(mask.view(np.int64)))
    torch.cuda.synchronize()
    kv.check()
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):
        rows = slice(b, b + 1)
        tree._check_rows(out[rows], lse[rows], q[rows], K[b], V[b], okt.visible(mask[rows], offs[b], n), scale, True)
    assert (out[B:] == tree.PAD).all() and (lse[B:] == tree.PAD).all()


@pytest.mark.parametrize("n,L", [(3, 700), (30, 2000)])
def test_sequences_of_one_page_table_row(n, L):
    """Several trees' queries on the same cached tokens: a table whose rows are one."""
    Hq, Hkv, D, page, B = 8, 1, 64, 64, 4
    r = np.random.default_rng(n)
    pages, table, K, V = _sequences(6, Hkv, D, page, [L])
    kv = _cache(Hq, Hkv, D, page_tokens=page, num_pages=pages.shape[0])
    q = r.standard_normal((B * n, Hq, D)).astype(np.float16)
    mask = np.concatenate([okt.masks(tree._parents(r, n), 1) for _ in range(B)])
    lens = [L - 7 * b for b in range(B)]
    dt = tree._i32(table).expand(B, -1)
    out, lse = tree._full((B * n, Hq, D), "float16"), tree._full((B * n, Hq), "float32")
    kv.attend(_dev(pages), _dev(q), tree._i32(lens), dt, out, lse=lse, q_start=tree._i32(tree._starts([n] * B)), max_q=n,
              tree=_dev(mask.view(np.int64)))
    kv.check()
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    kv.check()
    for b, m in enumerate(lens):
        rows = slice(b * n, (b + 1) * n)
        tree._check_rows(out[rows], lse[rows], q[rows], K[0][:m], V[0][:m], okt.visible(mask[rows], m - n, m), D ** -0.5, False)


def test_a_wide_star_of_rejected_drafts_takes_as_many_rounds():
    """255 siblings, all of them rejected: as many sums of one row."""
    kv = _cache(1, 1, 64)
    c = tree._verify_problem(12, [256, 200, 256], 3001, True, "star", gap=6.0, sharp=2.0)
    for children in (1, 255):
        got = tree._run_verify(kv, c, max_children=children)
        kv.check()
        tree._check_verify(got, c, least=1e-9)
