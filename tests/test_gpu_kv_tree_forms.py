"""GPU attention with a tree in the forms that tests/test_gpu_kv_tree.py does not reach (tests/test_kv_tree_bounds.py counts them)."""
import pytest

from tests import test_gpu_kv_tree as tree

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
