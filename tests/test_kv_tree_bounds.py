"""Workspace bounds of attention with a tree beside those without (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests.test_kv_tree_host import HEADS, ROOT, _plan, host  # noqa: F401


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("kvb") / "kvb.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "shard_decomposed_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "kv_tree_bounds_check.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for f in (lib.kvb_plain, lib.kvb_tree):
        f.argtypes = [ctypes.c_int] * 3 + [ctypes.c_int64] * 3 + [ctypes.c_int]
        f.restype = ctypes.c_int64
    return lib


@pytest.mark.parametrize("shape,most", [
    # Hq, Hkv, D, batch, max_q, max_kv; times the bound without trees
    ((64, 8, 128, 1, 1, 131072), 1.05), ((64, 8, 128, 16, 1, 8192), 1.25), ((64, 8, 128, 64, 1, 8192), 1.0),
    ((64, 8, 128, 1, 64, 131072), 1.05), ((64, 8, 128, 16, 64, 8192), 1.05), ((96, 8, 128, 1, 48, 131072), 1.05),
    ((32, 4, 64, 24, 25, 4099), 1.05)])
def test_workspaces_of_calls_without_trees_stay_near_what_those_need(bounds, shape, most):
    """kvc_attend_workspace holds calls of both kinds, so it is the larger of the two."""
    assert bounds.kvb_tree(*shape, 256) <= most * bounds.kvb_plain(*shape, 256)


@pytest.mark.parametrize("cus", [32, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_partials_hold_items_just_longer_than_their_runs(host, D, cus):  # noqa: F811
    """Lengths that leave every item a short last run, the most partials that there can be."""
    r = np.random.default_rng(D)
    full = 0.0
    for _ in range(400):
        Hq, Hkv = HEADS[r.integers(len(HEADS))]
        batch, max_q = (int(np.exp(r.uniform(0, np.log(top)))) for top in (512, 300))
        p = _plan(host, Hq, Hkv, D, batch, max_q, int(np.exp(r.uniform(5, 12))), int(r.integers(2)), cus)
        if p["slots"] == p["items"]:
            continue
        queries = np.full(batch, max_q, dtype=np.int32)
        at = lambda x: x.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))  # noqa: E731
        got = [ctypes.c_int64() for _ in range(3)]
        blocks = np.full(batch, int(p["least"]) + 1, dtype=np.int32)
        for _ in range(30):
            chunk = host.kvt_shared(Hkv, batch, at(blocks), at(queries), *[ctypes.byref(x) for x in got])
            work, partials, joins = (x.value for x in got)
            assert work <= p["slots"] and partials <= p["partials"] and joins <= min(p["items"], p["places"])
            full = max(full, partials / p["partials"])
            chunk = min(chunk, 1 << 20)
            blocks[:] = chunk + 1
            some = r.random(batch) < r.random()  # the others have one run
            blocks[some] = r.integers(0, chunk + 1, int(some.sum()))
            blocks[~some] += chunk * r.integers(0, 4)
    assert full > 0.75


def test_gpu_tests_reach_every_form_and_join(host):  # noqa: F811
    """Every (D, rows of a tile, several runs, joined by waves, output type) that some 20000 random calls are planned as."""
    from tests import test_gpu_kv_tree as one
    from tests import test_gpu_kv_tree_forms as more

    def form(Hq, Hkv, D, batch, max_q, max_kv, f32):
        p = _plan(host, Hq, Hkv, D, batch, max_q, max_kv, f32, 256)
        several = p["slots"] > p["items"]
        return D, p["rows"], several, several and p["join_rows"] > 0, f32
    reached = set()
    for Hq, Hkv, D, page, shape, max_kv in one.FORMS + more.FORMS:
        width = max(1, max(-(-n // page) for _, n in shape)) * page
        for f32 in (0, 1):
            reached.add(form(Hq, Hkv, D, len(shape), max(n for n, _ in shape), max_kv or width, f32))
    r, missing = np.random.default_rng(0), {}
    heads = [(64, 8), (96, 8), (8, 8), (1, 1), (12, 4), (32, 4), (16, 2), (40, 8), (24, 2), (32, 8), (16, 1), (64, 64)]
    for _ in range(20000):
        Hq, Hkv = heads[r.integers(len(heads))]
        shape = (Hq, Hkv, (64, 128, 256)[r.integers(3)], *(int(np.exp(r.uniform(0, np.log(top)))) for top in (200, 100, 9000)), int(r.integers(2)))
        if form(*shape) not in reached:
            missing[form(*shape)] = shape
    assert not missing
