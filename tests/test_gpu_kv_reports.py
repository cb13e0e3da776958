"""GPU tests of what kvc_check says: the very thing that a kernel met, also when many meet something at once."""
import re

import numpy as np
import pytest

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(gu.dev())


def _message(kv):
    import torch
    from shard_decomposed_gemm_amd import AgemmError
    torch.cuda.synchronize()
    with pytest.raises(AgemmError) as e:
        kv.check()
    kv.check()  # cleared
    return str(e.value)


@pytest.mark.parametrize("slot", [64, (1 << 32) + 5, (1 << 33), (1 << 34) + 7])
def test_report_of_slots_beyond_32_bits(slot):
    import torch
    from shard_decomposed_gemm_amd import KvCache
    kv = KvCache(1, 1, 64, page_tokens=32, num_pages=2)
    x = torch.ones(3, 1, 64, dtype=torch.float16, device=gu.dev())
    pages = kv.new_pages()
    kv.append(pages, k=x, v=x, slots=_dev(np.array([0, slot, 1])))
    assert f"token 1: slot {slot} past the last page (64 slots)" in _message(kv)
    kv.read(pages, _dev(np.array([0, 1, slot])), x, torch.empty_like(x))
    assert f"token 2: slot {slot} past the last page (64 slots)" in _message(kv)


def test_reports_of_many_workgroups_do_not_mix():
    """Every token has a slot or a position out of range that names the token; the message has to fit it."""
    import torch
    from shard_decomposed_gemm_amd import KvCache
    T, P, R = 4096, 2, 100
    kv = KvCache(2, 2, 64, page_tokens=32, num_pages=P)
    x = torch.ones(T, 2, 64, dtype=torch.float16, device=gu.dev())
    out, pages = torch.empty_like(x), kv.new_pages()
    t = np.arange(T)
    slots, pos = np.where(t % 3 == 0, t % 64, 1000 + 7 * t), np.where(t % 3 == 0, R + 11 * t, t % R)
    table = torch.ones(R, 64, device=gu.dev())
    for _ in range(20):
        kv.append(pages, q=x, k=x, v=x, slots=_dev(slots), positions=_dev(pos), rope=table, q_out=out)
        said = re.search(r"token (\d+): (slot|position) (\d+) ", _message(kv))
        at = int(said[1])
        assert (said[2], int(said[3])) == (("position", R + 11 * at) if at % 3 == 0 else ("slot", 1000 + 7 * at))


def test_reports_of_many_sequences_do_not_mix():
    import torch
    from shard_decomposed_gemm_amd import KvCache
    B = 400
    kv = KvCache(2, 1, 64, page_tokens=32, num_pages=2)
    q = torch.ones(B, 2, 64, dtype=torch.float16, device=gu.dev())
    out = torch.empty(B, 2, 64, device=gu.dev())
    b = np.arange(B)
    table = np.zeros((B, 3), dtype=np.int32)
    table[:, 1] = 5 + 3 * b  # a page id that names the sequence
    lens = np.where(b % 2 == 0, 96, 97 + b).astype(np.int32)  # or a length that does
    table[b % 2 == 1] = 0
    for _ in range(20):
        kv.attend(kv.new_pages(), q, _dev(lens), _dev(table), out)
        said = re.search(r"sequence (\d+): (page id|length) (\d+) ", _message(kv))
        at = int(said[1])
        assert (said[2], int(said[3])) == (("page id", 5 + 3 * at) if at % 2 == 0 else ("length", 97 + at))


def test_an_earlier_failed_hip_call_is_not_taken_for_the_cache_s():
    """A runtime call that failed before, somewhere else in the process, leaves its error for hipGetLastError; the
    cache's calls say what became of their own launches."""
    import ctypes

    import torch
    from shard_decomposed_gemm_amd import KvCache
    kv = KvCache(2, 1, 64, page_tokens=32, num_pages=64)
    x, out = torch.ones(3, 1, 64, dtype=torch.float16, device=gu.dev()), torch.empty(1, 2, 64, device=gu.dev())
    q, slots, pages = torch.ones(1, 2, 64, dtype=torch.float16, device=gu.dev()), _dev(np.arange(3)), kv.new_pages()
    table = torch.arange(64, dtype=torch.int32, device=gu.dev())[None]
    lens = torch.full((1,), 3, dtype=torch.int32, device=gu.dev())
    ws, back = kv.workspace(1, 1, 2048), torch.empty_like(x)
    torch.cuda.synchronize()
    hip = ctypes.CDLL([line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line][0])
    fail = lambda: hip.hipSetDevice(100000)  # noqa: E731 (refused)
    try:
        for call in (lambda: kv.append(pages, k=x, v=x, slots=slots), lambda: kv.read(pages, slots, back, torch.empty_like(x)),
                     lambda: kv.attend(pages, q, lens, table, out, workspace=ws)):
            assert fail() != 0
            call()
            assert hip.hipGetLastError() != 0  # and it is still there for whoever asks
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    kv.check()
    assert (out == 1).all() and (back == 1).all()
