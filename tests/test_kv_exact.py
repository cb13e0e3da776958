"""That the exact attention checks of tests/kv_exact.py see a block left out, taken twice or paired wrongly, on the CPU."""
import numpy as np
import pytest

from oracle import kv as okv
from tests import kv_exact as kx


def _outputs(shown, values):
    """Mean of the shown tokens' values and the log of their count."""
    n = shown.sum()
    return (values * shown[:, None]).sum(0)[None] / n, np.log(n)[None], np.array([n])


@pytest.mark.parametrize("D", [64, 128])
def test_hidden_tokens_have_no_weight(D):
    c = kx.Sequences(D, 2, D, 32, [300, 40])
    kn, ks, kb, vn, vs, vb = okv.unpack(c.pages, 2, D, 32)
    slot = (c.table[0, :10, None] * 32 + np.arange(32)).reshape(-1)[:300]
    K, V = okv.held(kn[slot], ks[slot], kb[slot]), okv.held(vn[slot], vs[slot], vb[slot])
    seen = np.array([0, 1, 33, 300])
    O, lse, _, _ = okv.attend(np.full((4, 6, D), -1.0), K, V, seen, kx.SCALE)
    want, count = c.rows(0, seen, 3)
    np.testing.assert_allclose(O, want, rtol=1e-12)
    assert kx.close(O, lse, want, count, True, 0).all()


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("L", [9000, 70000, 90000, 262144])
def test_a_wrong_block_shows(L, f32):
    """One block of 32 tokens left out, taken twice, or its values those of the next: each shows wherever it is."""
    D = 64
    c = kx.Sequences(3, 1, D, 64, [L])
    shown, values = c.shown[0][:, 0], c.values[0][:, 0].astype(np.int64)
    O, lse, n = _outputs(shown, values)
    rounded = (lambda o: o) if f32 else (lambda o: o.astype(np.float16).astype(np.float64))
    assert kx.close(rounded(O), lse, O, n, f32).all()
    for at in np.random.default_rng(L).integers(0, L // 32 - 1, 8):
        block = slice(32 * at, 32 * at + 32)
        without, twice = np.delete(np.arange(L), np.arange(L)[block]), np.concatenate([np.arange(L), np.arange(L)[block]])
        for take in (without, twice):
            wrong, l, _ = _outputs(shown[take], values[take])
            assert not kx.close(rounded(wrong), l, O, n, f32).all()
        if f32:  # a swap leaves the count, and moves the means by less than binary16 holds
            swapped = values.copy()
            swapped[block] = values[block.stop:block.stop + 32]
            wrong, l, _ = _outputs(shown, swapped)
            assert not kx.close(wrong, l, O, n, f32).all()
