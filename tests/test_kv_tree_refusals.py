"""Calls with trees that have no meaning are refused (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from shard_decomposed_gemm_amd import agemm, kvc
from tests.test_kv_tree_host import A, ROOT, host  # noqa: F401


@pytest.fixture(scope="module")
def apart(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("kva") / "kva.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "shard_decomposed_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "kv_apart_check.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.kva_tree.argtypes = [ctypes.POINTER(kvc.TreeArgs), ctypes.c_char_p]
    lib.kva_verify.argtypes = [ctypes.POINTER(kvc.VerifyArgs), ctypes.c_void_p, ctypes.c_int64, ctypes.c_char_p]
    lib.kva_commit.argtypes = [ctypes.POINTER(kvc.CommitArgs), ctypes.c_char_p]
    return lib


@pytest.mark.parametrize("max_q,words,code", [
    (1, 1, agemm.OK), (64, 1, agemm.OK), (65, 1, agemm.EINVAL), (128, 2, agemm.OK), (129, 2, agemm.EINVAL),
    (1024, 16, agemm.OK), (1025, 16, agemm.EINVAL), (1 << 23, 16, agemm.EINVAL)])
def test_masks_hold_every_query(host, max_q, words, code):  # noqa: F811
    """A row of more nodes than its mask has bits could not see itself."""
    why = ctypes.create_string_buffer(256)
    assert host.kvt_mask(kvc.AttendArgs(batch=2, tokens=5, causal=1, max_q=max_q), A, words, why) == code
    assert (b"max_q" in why.value) == (code != agemm.OK)


def _spread(fields, **sizes):
    """Addresses of arrays one right behind the other, in the order of `sizes`."""
    at, out = A, {}
    for name, size in sizes.items():
        out[name] = at
        at += size
    return {**fields, **out}


T, B, V = 20, 3, 50
TREE = _spread(dict(batch=B, tokens=T, max_q=10, table_stride=6, table_width=4, mask_words=2), mask=T * 16, positions=T * 8,
               slots=T * 8, total_len=B * 4, q_start=(B + 1) * 4, kv_len=B * 4, parent=T * 4, page_table=(2 * 6 + 4) * 4)
VERIFY = _spread(dict(batch=B, tokens=T, max_q=10, p_stride=V + 2, q_stride=0, vocab=V, max_children=1), path=T * 4, count=B * 4,
                 next=B * 8, q_start=(B + 1) * 4, parent=T * 4, token=T * 8, u=T * 4, p=((T - 1) * (V + 2) + V) * 4, q=V * 4)
COMMIT = _spread(dict(batch=B, tokens=T, max_q=10, table_stride=0, table_width=4), new_len=B * 4, q_start=(B + 1) * 4, kv_len=B * 4,
                 path=T * 4, count=B * 4, page_table=16)


def _apart(apart, kind, fields, ws=(0, 0)):
    why = ctypes.create_string_buffer(256)
    rc = {"tree": lambda: apart.kva_tree(kvc.TreeArgs(**fields), why),
          "verify": lambda: apart.kva_verify(kvc.VerifyArgs(**fields), *ws, why),
          "commit": lambda: apart.kva_commit(kvc.CommitArgs(**fields), why)}[kind]()
    assert (rc == agemm.EINVAL) == (b"must lie apart" in why.value)
    return rc


@pytest.mark.parametrize("kind,fields,outputs", [
    ("tree", TREE, ("mask", "positions", "slots", "total_len")), ("verify", VERIFY, ("path", "count", "next")),
    ("commit", COMMIT, ("new_len",))])
def test_outputs_lie_apart_from_all_that_is_read(apart, kind, fields, outputs):
    """One right behind the other is apart; the same array, the last element of one and the first of another are not."""
    arrays = [k for k, v in fields.items() if v >= A]
    assert _apart(apart, kind, fields) == agemm.OK
    for out in outputs:
        assert _apart(apart, kind, {**fields, out: None}) == agemm.OK
        for other in arrays:
            if other != out:
                assert _apart(apart, kind, {**fields, other: fields[out]}) == agemm.EINVAL, (out, other)
                assert _apart(apart, kind, {**fields, out: fields[other]}) == agemm.EINVAL, (out, other)
    for left, right in zip(arrays, arrays[1:]):  # moved into its neighbour by an element
        step = 8 if left in ("mask", "positions", "slots", "next", "token") else 4
        if left in outputs or right in outputs:
            assert _apart(apart, kind, {**fields, left: fields[left] + step}) == agemm.EINVAL, (left, right)


def test_workspace_of_a_verification_lies_apart(apart):
    end = VERIFY["q"] + V * 4
    assert _apart(apart, "verify", VERIFY, (end, 4096)) == agemm.OK
    assert _apart(apart, "verify", VERIFY, (end - 4, 4096)) == agemm.EINVAL
    assert _apart(apart, "verify", VERIFY, (A - 4096, 4096)) == agemm.OK
    assert _apart(apart, "verify", VERIFY, (A - 4096, 4097)) == agemm.EINVAL


def test_empty_arrays_lie_apart(apart):
    assert _apart(apart, "tree", {**TREE, "tokens": 0, **{k: A for k in ("mask", "positions", "slots", "parent")}}) == agemm.OK
    assert _apart(apart, "verify", {**VERIFY, "tokens": 0, "path": VERIFY["u"]}) == agemm.OK


def test_extents_of_the_widest_strides_do_not_overflow(apart):
    """Rows 2^40 elements apart, 2^23 of them: past 2^63 bytes."""
    at = 1 << 45
    far = {**VERIFY, "tokens": 1 << 23, "p_stride": 1 << 40, "q": None, **{k: at - (i + 1 << 26) for i, k in enumerate(
        ("path", "count", "next", "q_start", "parent", "token", "u"))}, "p": at}
    assert _apart(apart, "verify", far) == agemm.OK
    assert _apart(apart, "verify", {**far, "next": at + (1 << 50)}) == agemm.EINVAL
    assert _apart(apart, "verify", {**far, "p_stride": 0, "next": at + (1 << 50)}) == agemm.OK
