"""GPU calls with trees whose outputs overlap what is read: refused, nothing launched (tests/test_kv_tree_refusals.py has every pair)."""
import pytest

from tests import gpu_util as gu
from tests.test_gpu_kv import _cache
from tests.test_gpu_kv_tree import _full, _i32

pytestmark = pytest.mark.gpu


def test_overlapping_outputs_are_refused():
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    kv = _cache(2, 1, 64, page_tokens=32, num_pages=4)
    parent, starts, lens, table = _i32([-1, 0, 0]), _i32([0, 3]), _i32([5]), _i32([[0, 1]])
    token, u, p = _full((3,), "int64", 0), torch.zeros(3, device=gu.dev()), torch.ones(3, 10, device=gu.dev())
    path, count, nxt = _i32([0, -1, -1]), _i32([1]), _full((1,), "int64", 0)
    longs, ws = _full((9,), "int64", 7), kv.verify_workspace(1, 10)
    for call in (
            lambda: kv.verify(token, parent, starts, p, u, parent, count, nxt, 3),
            lambda: kv.verify(token, parent, starts, p, u, path, path[2:], nxt, 3),
            lambda: kv.verify(token, parent, starts, p, u, path, count, token[:1], 3),
            lambda: kv.verify(token, parent, starts, p, u, path, count, ws[:8].view(torch.int64), 3, workspace=ws),
            lambda: kv.tree(parent, starts, lens, table, 3, longs[:3, None], positions=longs[2:5]),
            lambda: kv.tree(parent, starts, lens, table, 3, longs[:3, None], slots=longs[:3]),
            lambda: kv.tree(parent, starts, lens, table, 3, longs[:3, None], total_len=parent[:1]),
            lambda: kv.commit([], starts, lens, path, count, table, 3, new_len=path[1:2])):
        with pytest.raises(AgemmError, match="must lie apart"):
            call()
    torch.cuda.synchronize()
    assert (longs == 7).all() and parent.tolist() == [-1, 0, 0] and path.tolist() == [0, -1, -1] and count.tolist() == [1]
    kv.tree(parent, starts, lens, table, 3, longs[:3, None], positions=longs[3:6], slots=longs[6:])  # neighbours
    kv.verify(token, parent, starts, p, u, path, count, nxt, 3)
    torch.cuda.synchronize()
    kv.check()
    assert longs.tolist() == [1, 3, 5, 5, 6, 6, 5, 6, 7] and count.tolist()[0] >= 1
