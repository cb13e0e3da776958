"""Functions that the key/value cache's kernels share with its host library, on the CPU at the ends of their ranges."""
import ctypes
import os
import re
import shutil
import subprocess

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
    lib.kvu_needs.argtypes, lib.kvu_needs.restype = [ctypes.c_int] * 3 + [ctypes.c_int64] * 3 + [ctypes.c_int], ctypes.c_int64
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
