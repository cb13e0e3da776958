"""Functions that the key/value cache's kernels share with its host library, on the CPU at the ends of their ranges."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "shard_decomposed_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("kvu") / "kvu.so")
    subprocess.run([gxx, "-O2", "-fwrapv", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "kv_units_check.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for f in (lib.kvu_workspace, lib.kvu_needs):
        f.argtypes, f.restype = [ctypes.c_int] * 3 + [ctypes.c_int64] * 3 + [ctypes.c_int], ctypes.c_int64
    lib.kvu_report.argtypes = [ctypes.c_uint32] + [ctypes.c_int64] * 4 + [ctypes.c_char_p]
    lib.kvu_report.restype = None
    return lib


def test_blocks_of_every_length_that_fits_32_bits(units):
    top = (1 << 31) - 1
    for n in [0, 1, 31, 32, 33, 63, 64, 65, 1 << 30, *range(top - 70, top + 1)]:
        assert units.kvu_blocks(n) == -(-n // 32), n


def test_kernels_count_blocks_with_the_shared_function():
    source = open(os.path.join(CSRC, "kv_attend.hip")).read()
    assert "kv_blocks(" in source and not re.search(r"\+ 31\)?\s*(>> 5|/ 32)", source)


@pytest.mark.parametrize("Hq,Hkv,D", [(64, 8, 128), (96, 96, 128), (16, 2, 256), (64, 1, 64)])
def test_plan_of_an_empty_batch(units, Hq, Hkv, D):
    for max_q in (1, 3, 700):
        for max_kv in (1, 1024, 1025, 262144, (1 << 31) - 1):
            assert units.kvu_needs(Hq, Hkv, D, 0, max_q, max_kv, 256) == 0


# ---------------------------------------------------------------- the workspace of calls within bounds

def _sizes(top):
    """Every size up to 70, then some of each octave and both sides of its ends, up to top."""
    few = list(range(1, 71))
    for p in range(6, 32):
        few += [(1 << p) + d for d in (-1, 0, 1)] + [3 << (p - 1), (5 << (p - 2)) + 1]
    return sorted({x for x in few if x <= top} | {top})


@pytest.mark.parametrize("cus", [256, 32, 304])
@pytest.mark.parametrize("Hq,Hkv,D", [(64, 8, 128), (32, 8, 128), (96, 8, 128), (96, 96, 128), (12, 1, 128), (1, 1, 64),
                                      (17, 1, 64), (32, 4, 64), (16, 2, 256), (8, 8, 256), (40, 2, 128), (1024, 1024, 64),
                                      (600, 600, 128), (1024, 1, 64)])
def test_workspace_of_bounds_holds_every_smaller_call(units, Hq, Hkv, D, cus):
    """A server's workspace, made once for its largest batch, chunk and length, serves its smaller steps too."""
    r = np.random.default_rng(Hq + D)
    for batch, max_q, max_kv in ((256, 1, 8192), (64, 1, 8192), (8, 2048, 8192), (4, 2048, 16384), (512, 64, 40000),
                                 (700, 4, 1 << 20), (1, 1, 262144), (3, 40, 1000), (2, 5, (1 << 31) - 1), (8192, 700, 33),
                                 (1, 1, 1), (0, 1, 8192)):
        size = units.kvu_workspace(Hq, Hkv, D, batch, max_q, max_kv, cus)
        pick = lambda top, n: r.choice(_sizes(top), min(n, len(_sizes(top))), replace=False).tolist() + [top]  # noqa: E731
        worst = 0
        for b in pick(batch, 60) if batch else [0]:
            for q in pick(max_q, 24):
                for kv in pick(max_kv, 24):
                    worst = max(worst, units.kvu_needs(Hq, Hkv, D, b, q, kv, cus))
        assert worst <= size, (batch, max_q, max_kv)
        # and it is no more than calls within the bounds come to, but for a factor
        assert size <= 4 * worst + (1 << 20), (batch, max_q, max_kv, worst, size)
        for b, q, kv in ((batch // 2, max_q, max_kv), (batch, max(1, max_q // 3), max_kv), (batch, max_q, max(1, max_kv - 1))):
            assert units.kvu_workspace(Hq, Hkv, D, b, q, kv, cus) <= size


@pytest.mark.parametrize("Hq,Hkv,D", [(64, 8, 128), (96, 96, 128), (1, 1, 64), (16, 2, 256), (1024, 1, 64)])
def test_plan_of_lengths_beyond_the_longest(units, Hq, Hkv, D):
    """max_kv is only what to expect: beyond the longest length it stands for that, up to the largest number."""
    for batch, max_q in ((1, 1), (3, 40), (400, 2), (8, 700), (1 << 23, 1 << 23)):
        for f in (units.kvu_needs, units.kvu_workspace):
            want = f(Hq, Hkv, D, batch, max_q, 1 << 31, 256)
            assert want >= 0
            for max_kv in ((1 << 31) + 1, 1 << 40, (1 << 63) - 40, (1 << 63) - 1):
                assert f(Hq, Hkv, D, batch, max_q, max_kv, 256) == want


# ---------------------------------------------------------------- reports

def test_report_says_what_was_met(units):
    buf = ctypes.create_string_buffer(256)

    def text(code, index, seen):
        units.kvu_report(code, index, seen, 1 << 40, 77, buf)
        return buf.value.decode()

    top = (1 << 23) - 1
    for at in (0, 5, 4097, top):
        for v in (1 << 40, (1 << 32) + 5, (1 << 31), (1 << 35) - 2, 64):
            said = f"from {(1 << 35) - 1}" if v >= (1 << 35) - 1 else v
            assert text(1, at, v) == f"token {at}: slot {said} past the last page ({1 << 40} slots)"
            assert text(2, at, v) == f"token {at}: position {said} outside the rotation table"
        for v in (-1, -5, -(1 << 31) - 1, -(1 << 35) + 1):
            assert text(2, at, v) == f"token {at}: position {v} outside the rotation table"
        assert text(2, at, -(1 << 63)) == f"token {at}: position up to {-(1 << 35)} outside the rotation table"
        assert f"token {at}: " in text(3, at, 1023) and "kv head 1023" in text(3, at, 1023)
        for v in (-(1 << 31), -1, 77, (1 << 31) - 1):
            assert text(4, at, v) == f"sequence {at}: page id {v} outside the cache (77 pages)"
            assert text(5, at, v).startswith(f"sequence {at}: length {v} ")
        for v in (-(1 << 32) + 1, -1, (1 << 32) - 1):
            assert text(6, at, v).startswith(f"sequence {at}: {v} query rows")
    assert "unknown case 0" in text(0, 0, 0)
