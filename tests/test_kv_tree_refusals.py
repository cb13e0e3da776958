"""Calls with trees that have no meaning are refused (no GPU)."""
import ctypes

import pytest

from shard_decomposed_gemm_amd import agemm, kvc
from tests.test_kv_tree_host import A, host  # noqa: F401


@pytest.mark.parametrize("max_q,words,code", [
    (1, 1, agemm.OK), (64, 1, agemm.OK), (65, 1, agemm.EINVAL), (128, 2, agemm.OK), (129, 2, agemm.EINVAL),
    (1024, 16, agemm.OK), (1025, 16, agemm.EINVAL), (1 << 23, 16, agemm.EINVAL)])
def test_masks_hold_every_query(host, max_q, words, code):  # noqa: F811
    """A row of more nodes than its mask has bits could not see itself."""
    why = ctypes.create_string_buffer(256)
    assert host.kvt_mask(kvc.AttendArgs(batch=2, tokens=5, causal=1, max_q=max_q), A, words, why) == code
    assert (b"max_q" in why.value) == (code != agemm.OK)
