"""GPU tests of what kvc_append stores, bit for bit (tests/kv_bits.py): the 4-bit form that binary64 gives."""
import numpy as np
import pytest

from oracle import kv as okv
from tests import gpu_util as gu
from tests import kv_bits as kb

pytestmark = pytest.mark.gpu


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(gu.dev())


def _append(k, v, page, **kw):
    """What the pages hold of keys and values (T, Hkv, D): kn, ks, kb, vn, vs, vb."""
    import torch
    from shard_decomposed_gemm_amd import KvCache
    T, Hkv, D = k.shape
    P = -(-T // page)
    kv = KvCache(Hkv, Hkv, D, page_tokens=page, num_pages=P)
    pages, slots = kv.new_pages(), np.random.default_rng(T).permutation(P * page)[:T]
    kv.append(pages, k=_dev(k), v=_dev(v), slots=_dev(slots), **kw)
    torch.cuda.synchronize()
    kv.check()
    return [y[slots] for y in okv.unpack(pages.cpu().numpy(), Hkv, D, page)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (7, 5), (300, 3), (1500, 8)])
def test_values_and_plain_keys_are_the_oracle_s_bits(T, Hkv, D):
    x = kb.rows(T + D, 2 * T * Hkv, D)[:2 * T * Hkv]
    x = np.random.default_rng(D).permutation(x).reshape(2, T, Hkv, D)
    kn, ks, kb_, vn, vs, vb = _append(x[0], x[1], 64)
    assert kb.exact(x[0], kn, ks, kb_).all()
    assert kb.exact(x[1], vn, vs, vb).all()


@pytest.mark.parametrize("D,R,interleaved,norm", [
    (64, 64, False, True), (64, 32, True, False), (64, 0, False, True), (128, 128, False, True), (128, 128, True, True),
    (128, 48, False, False), (256, 256, False, False), (256, 64, False, True)])
def test_normed_and_rotated_keys_are_what_binary64_gives(D, R, interleaved, norm):
    """Other bits only where the binary64 number lies within binary64's error of a border between two."""
    T, Hkv, length = 6000, 4, 20000
    r = np.random.default_rng(D + R)
    k = (r.standard_normal((T, Hkv, D)) * np.exp2(r.integers(-3, 4, (T, Hkv, 1)))).astype(np.float16)
    w = (1 + 0.3 * r.standard_normal(D)).astype(np.float16)
    pos = r.integers(0, length, T)
    kw, y = {}, k.astype(np.float64)
    if norm:
        kw, y = dict(k_norm=_dev(w), eps=2.0 ** -20), okv.norm(y, w, 2.0 ** -20)
    if R:
        a = np.arange(length)[:, None] * 10000.0 ** (-2 * np.arange(R // 2) / R)
        table = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
        kw.update(rope=_dev(table), positions=_dev(pos), interleaved=interleaved)
        y = okv.rope(y, table[pos], interleaved)
    kn, ks, kb_, vn, vs, vb = _append(k, k, 32, **kw)
    assert kb.near(y, kn, ks, kb_).all()
    assert kb.exact(k, vn, vs, vb).all()
