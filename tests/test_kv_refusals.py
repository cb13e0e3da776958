"""Refusals of the key/value cache's calls that came with their limits, on the CPU."""
import ctypes

import pytest

from shard_decomposed_gemm_amd import agemm
from tests.test_kv_host import SHAPE, _attend, host  # noqa: F401 (a fixture)


@pytest.mark.parametrize("scale,code", [
    (2.0 ** 127, agemm.EINVAL), (-(2.0 ** 127), agemm.EINVAL), (3e38, agemm.EINVAL), (1.99 * 2.0 ** 126, agemm.OK),
    (-(2.0 ** 126), agemm.OK), (0.0, agemm.OK), (2.0 ** -149, agemm.OK)])
def test_attend_scale_leaves_room_for_the_factor_of_log_2(host, scale, code):  # noqa: F811
    why = ctypes.create_string_buffer(256)
    assert host.kvh_attend(*SHAPE, 0x10000, _attend(scale=scale), 0, None, 0, why) == code
