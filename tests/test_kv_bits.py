"""That the bit-for-bit checks of tests/kv_bits.py see a quantiser's mistakes, planted here on the CPU."""
import numpy as np
import pytest

from oracle import kv as okv
from tests import kv_bits as kb


def _binary32(x, divide=True, ties=np.rint):
    """The 4-bit form with binary32 arithmetic and no care at the borders."""
    x = np.asarray(x, dtype=np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    s = ((hi - lo) * np.float32(1 / 15) if not divide else (hi - lo) / np.float32(15)).astype(np.float16)
    sf = s.astype(np.float32)
    b = (lo - np.float32(16) * sf).astype(np.float16)
    step = np.where(sf > 0, sf, 1)
    t = (x - b.astype(np.float32)) / step if divide else (x - b.astype(np.float32)) * (np.float32(1) / step)
    return np.clip(np.where(sf > 0, ties(t) - 16, 0), 0, 15).astype(np.uint8), s, b


@pytest.mark.parametrize("D", [64, 128, 256])
def test_exact_rows_pass_the_oracle_and_show_mistakes(D):
    x = kb.rows(D, 1200, D)
    assert np.isfinite(x.astype(np.float64)).all() and (np.abs(x.astype(np.float64)) <= okv.LIMIT).all()
    n, s, b, _ = okv.quantise(x)
    assert kb.exact(x, n, s, b).all() and kb.near(x.astype(np.float64), n, s, b).all()
    up, down = (lambda t: np.floor(t + np.float32(0.5))), (lambda t: np.ceil(t - np.float32(0.5)))
    for wrong in (_binary32(x, divide=False), _binary32(x, ties=up), _binary32(x, ties=down)):
        assert not kb.exact(x, *wrong).all()
    # one unit of s or b, one nibble
    for change in ((n, np.nextafter(s, np.float16(np.inf)), b), (n, s, np.nextafter(b, np.float16(0))), (n ^ 1, s, b)):
        assert not kb.exact(x, *change).all()


def _normed_and_rotated(x, w, table, interleaved):
    """Norm and rotation in binary32."""
    x, w = x.astype(np.float32), w.astype(np.float32)
    x = x * (np.float32(1) / np.sqrt((x * x).mean(-1, keepdims=True) + np.float32(2.0 ** -20))) * w
    R = x.shape[-1]
    cos, sin = table[:, None, :R // 2], table[:, None, R // 2:]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y = np.empty_like(x)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    return y


@pytest.mark.parametrize("D,interleaved", [(64, True), (128, False), (256, False)])
def test_normed_and_rotated_rows_show_binary32(D, interleaved):
    r = np.random.default_rng(D)
    x = r.standard_normal((24000, 1, D)).astype(np.float16)
    w = (1 + 0.3 * r.standard_normal(D)).astype(np.float16)
    a = r.uniform(0, 6.3, (24000, D // 2))
    table = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    y = okv.rope(okv.norm(x, w, 2.0 ** -20), table, interleaved)
    n, s, b, _ = okv.quantise(y)
    assert kb.near(y, n, s, b).all()
    assert kb.near(y, *okv.quantise(y * (1 + 1e-14))[:3]).all()
    z = _normed_and_rotated(x, w, table, interleaved)
    np.testing.assert_allclose(z, y, atol=1e-5)
    assert not kb.near(y, *_binary32(z)).all()
