"""Drafted tokens in a tree on the CPU (no GPU): the oracle's pins, refusals, plans, reports.

tests/kv_tree_check.cpp compiles the host library's own argument checks
(csrc/kv_checks.h) with g++, so that every refusal is tested before anything
could be launched.
"""
import ctypes
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import kvtree as okt
from shard_decomposed_gemm_amd import agemm, kvc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("kvt") / "kvt.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "shard_decomposed_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "kv_tree_check.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_char_p
    lib.kvt_mask.argtypes = [ctypes.POINTER(kvc.AttendArgs), vp, i32, st]
    lib.kvt_tree.argtypes = [ctypes.POINTER(kvc.TreeArgs), st]
    lib.kvt_verify.argtypes = [ctypes.POINTER(kvc.VerifyArgs), i64, vp, i64, st]
    lib.kvt_commit.argtypes = [ctypes.c_int, vp, i32, ctypes.POINTER(kvc.CommitArgs), st]
    lib.kvt_commit_piece.argtypes = [ctypes.c_int, i64]
    lib.kvt_verify_plan.argtypes = [i64, i64, ctypes.c_int, i64, ctypes.c_int, ctypes.POINTER(i32)]
    lib.kvt_verify_bound.argtypes = [i64, i64, ctypes.c_int]
    lib.kvt_verify_bound.restype = i64
    ints, longs = ctypes.POINTER(i32), ctypes.POINTER(i64)
    lib.kvt_plan.argtypes = [ctypes.c_int] * 3 + [i64] * 3 + [ctypes.c_int] * 2 + [longs]
    lib.kvt_plan.restype = None
    lib.kvt_bound.argtypes = [ctypes.c_int] * 3 + [i64] * 3 + [ctypes.c_int]
    lib.kvt_bound.restype = i64
    lib.kvt_shared.argtypes = [ctypes.c_int, ctypes.c_int, ints, ints, longs, longs, longs]
    lib.kvt_report.argtypes = [ctypes.c_uint32, i64, i64, st]
    return lib


# ---------------------------------------------------------------- interface

STRUCTS = {"kvc_tree_args": (kvc.TreeArgs, kvc._pack_tree), "kvc_verify_args": (kvc.VerifyArgs, kvc._pack_verify),
           "kvc_commit_args": (kvc.CommitArgs, kvc._pack_commit)}


def test_argument_structs_are_the_headers(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kvcache.h"', "int main(void) {"]
    want = []
    for name, (st, pack) in STRUCTS.items():
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        lines += [f'  printf("%zu\\n", offsetof({name}, {f[0]}));' for f in st._fields_]
        want += [ctypes.sizeof(st)] + [getattr(st, f[0]).offset for f in st._fields_]
        values = list(range(1, len(st._fields_) + 1))
        got = st.from_buffer_copy(pack(*values).ljust(ctypes.sizeof(st), b"\0"))
        assert [getattr(got, f[0]) for f in st._fields_] == values
    src, exe = tmp_path / "s.c", str(tmp_path / "s")
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    assert [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()] == want


def test_null_contexts_are_refused():
    lib = kvc.load()
    n = ctypes.c_int64()
    assert lib.kvc_tree(None, None, None) == agemm.EINVAL
    assert lib.kvc_attend_tree(None, None, None, None, 1, None, 0, None) == agemm.EINVAL
    assert lib.kvc_verify(None, None, None, 0, None) == agemm.EINVAL
    assert lib.kvc_verify_workspace(None, 1, 100, ctypes.byref(n)) == agemm.EINVAL
    assert lib.kvc_commit(None, None, 0, None, None) == agemm.EINVAL


# ---------------------------------------------------------------- refusals

NOTHING = -1


def _tree(**change):
    a = dict(batch=2, max_q=10, tokens=20, q_start=A, kv_len=A + 64, parent=A, page_table=A, table_stride=4, table_width=4,
             mask_words=1, mask=A, positions=A, slots=A, total_len=A + 128)
    return kvc.TreeArgs(**{**a, **change})


@pytest.mark.parametrize("change,code", [
    ({}, agemm.OK), (dict(positions=None, slots=None, total_len=None, page_table=None), agemm.OK),
    (dict(batch=0), agemm.OK), (dict(batch=0, tokens=0), NOTHING), (dict(tokens=0, total_len=None), NOTHING),
    (dict(tokens=0), agemm.OK), (dict(tokens=0, parent=None, mask=None), agemm.OK),
    (dict(max_q=64), agemm.OK), (dict(max_q=65), agemm.EINVAL), (dict(max_q=1024, mask_words=16), agemm.OK),
    (dict(max_q=1025, mask_words=17), agemm.EINVAL), (dict(mask_words=0), agemm.EINVAL), (dict(max_q=0), agemm.EINVAL),
    (dict(batch=-1), agemm.EINVAL), (dict(tokens=-1), agemm.EINVAL), (dict(tokens=(1 << 23) + 1), agemm.ESHAPE),
    (dict(batch=(1 << 20) + 1), agemm.ESHAPE), (dict(q_start=None), agemm.EINVAL), (dict(kv_len=None), agemm.EINVAL),
    (dict(parent=None), agemm.EINVAL), (dict(mask=None), agemm.EINVAL), (dict(page_table=None), agemm.EINVAL),
    (dict(table_stride=3), agemm.EINVAL), (dict(table_stride=0), agemm.OK), (dict(table_width=0), agemm.EINVAL),
    (dict(table_stride=-4), agemm.EINVAL), (dict(total_len=A + 64), agemm.EINVAL), (dict(total_len=A), agemm.EINVAL),
    (dict(mask=A + 4), agemm.EINVAL), (dict(slots=A + 4), agemm.EINVAL), (dict(parent=A + 2), agemm.EINVAL),
    (dict(page_table=A + 2), agemm.EINVAL)])
def test_tree_refusals(host, change, code):
    why = ctypes.create_string_buffer(256)
    assert host.kvt_tree(_tree(**change), why) == code
    assert bool(why.value) == (code > 0)


def test_tree_without_arguments(host):
    assert host.kvt_tree(None, ctypes.create_string_buffer(256)) == agemm.EINVAL


@pytest.mark.parametrize("causal,batch,mask,words,code", [
    (1, 2, A, 1, agemm.OK), (1, 2, A, 16, agemm.OK), (1, 2, A, 17, agemm.EINVAL), (1, 2, A, 0, agemm.EINVAL),
    (0, 2, A, 1, agemm.EINVAL), (1, 2, None, 1, agemm.EINVAL), (1, 0, None, 1, agemm.OK), (1, 2, A + 4, 1, agemm.EINVAL)])
def test_mask_refusals(host, causal, batch, mask, words, code):
    assert host.kvt_mask(kvc.AttendArgs(batch=batch, tokens=5, causal=causal), mask, words,
                         ctypes.create_string_buffer(256)) == code


def _verify(**change):
    a = dict(batch=2, max_q=10, tokens=20, q_start=A, parent=A, token=A, p=A, q=A, p_stride=100, q_stride=100, vocab=100,
             u=A, max_children=1, path=A, count=A, next=A)
    return kvc.VerifyArgs(**{**a, **change})


@pytest.mark.parametrize("change,code", [
    ({}, agemm.OK), (dict(q=None, q_stride=3), agemm.OK), (dict(batch=0), NOTHING), (dict(p_stride=0, q_stride=0), agemm.OK),
    (dict(p_stride=99), agemm.EINVAL), (dict(q_stride=99), agemm.EINVAL), (dict(p_stride=-100), agemm.EINVAL),
    (dict(p_stride=101), agemm.OK), (dict(vocab=0), agemm.ESHAPE), (dict(vocab=(1 << 28) + 1, p_stride=1 << 29), agemm.ESHAPE),
    (dict(max_q=0), agemm.EINVAL), (dict(max_q=1025), agemm.EINVAL), (dict(max_children=0), agemm.EINVAL),
    (dict(q_start=None), agemm.EINVAL), (dict(parent=None), agemm.EINVAL), (dict(token=None), agemm.EINVAL),
    (dict(p=None), agemm.EINVAL), (dict(u=None), agemm.EINVAL), (dict(path=None), agemm.EINVAL),
    (dict(count=None), agemm.EINVAL), (dict(next=None), agemm.EINVAL), (dict(tokens=0, p=None, path=None), agemm.OK),
    (dict(token=A + 4), agemm.EINVAL), (dict(next=A + 4), agemm.EINVAL), (dict(p=A + 2), agemm.EINVAL),
    (dict(batch=-1), agemm.EINVAL), (dict(batch=(1 << 20) + 1), agemm.ESHAPE)])
def test_verify_refusals(host, change, code):
    why = ctypes.create_string_buffer(256)
    assert host.kvt_verify(_verify(**change), 4096, A, 4096, why) == code
    assert bool(why.value) == (code > 0)


def test_verify_workspace_refusals(host):
    why = ctypes.create_string_buffer(256)
    assert host.kvt_verify(_verify(), 4096, A, 4095, why) == agemm.EINVAL
    assert host.kvt_verify(_verify(), 4096, None, 4096, why) == agemm.EINVAL
    assert host.kvt_verify(_verify(), 4096, A + 8, 4096, why) == agemm.EINVAL
    assert host.kvt_verify(None, 0, A, 4096, why) == agemm.EINVAL


def _commit(**change):
    a = dict(batch=2, max_q=10, tokens=20, q_start=A, kv_len=A + 64, path=A + 128, count=A + 256, page_table=A,
             table_stride=4, table_width=4, new_len=A + 320)
    return kvc.CommitArgs(**{**a, **change})


def _pointers(*at):
    return (ctypes.c_void_p * max(1, len(at)))(*at)


@pytest.mark.parametrize("change,pages,code", [
    ({}, [A], agemm.OK), ({}, [A, 2 * A], agemm.OK), ({}, [A, 2 * A, A], agemm.EINVAL), ({}, [A, 0], agemm.EINVAL),
    ({}, [A + 8], agemm.EINVAL), ({}, [], agemm.OK), (dict(new_len=None), [], NOTHING), (dict(new_len=None), [A], agemm.OK),
    (dict(batch=0), [A], NOTHING), (dict(tokens=0, path=None), [A], agemm.OK), (dict(path=None), [A], agemm.EINVAL),
    (dict(count=None), [A], agemm.EINVAL), (dict(kv_len=None), [A], agemm.EINVAL), (dict(q_start=None), [A], agemm.EINVAL),
    (dict(page_table=None), [A], agemm.EINVAL), (dict(table_stride=3), [A], agemm.EINVAL),
    (dict(new_len=A + 64), [A], agemm.EINVAL), (dict(new_len=A + 256), [A], agemm.EINVAL), (dict(new_len=A), [A], agemm.EINVAL),
    (dict(max_q=1025), [A], agemm.EINVAL), (dict(path=A + 130), [A], agemm.EINVAL), (dict(tokens=-1), [A], agemm.EINVAL)])
def test_commit_refusals(host, change, pages, code):
    why = ctypes.create_string_buffer(256)
    assert host.kvt_commit(2, _pointers(*pages), len(pages), _commit(**change), why) == code
    assert bool(why.value) == (code > 0)


def test_commit_refusals_of_counts(host):
    why = ctypes.create_string_buffer(256)
    assert host.kvt_commit(2, _pointers(A), -1, _commit(), why) == agemm.EINVAL
    assert host.kvt_commit(2, None, 1, _commit(), why) == agemm.EINVAL
    assert host.kvt_commit(2, _pointers(*(A + 16 * i for i in range(1024))), 1024, _commit(), why) == agemm.OK
    assert host.kvt_commit(2, _pointers(A), 1025, _commit(), why) == agemm.EINVAL
    assert host.kvt_commit(1024, _pointers(A), 1, _commit(batch=(1 << 15) + 1), why) == agemm.ESHAPE
    assert host.kvt_commit(2, _pointers(A), 1, None, why) == agemm.EINVAL


# ---------------------------------------------------------------- plans

def test_commit_launches_stay_below_2_to_32_threads(host):
    for Hkv in (1, 8, 96, 1024):
        for batch in (1, 7, 1000, (1 << 25) // Hkv):
            n = host.kvt_commit_piece(Hkv, batch)
            assert 1 <= n <= 64 and batch * Hkv * n * 64 < 1 << 32


@pytest.mark.parametrize("cus", [32, 256, 304])
def test_verify_plans_cover_the_vocabulary_within_their_bound(host, cus):
    out = (ctypes.c_int32 * 3)()
    for batch in (1, 2, 3, 5, 16, 17, 64, 100, 1023, 1024, 1025, 5000, 1 << 20):
        for vocab in (1, 2, 1023, 1024, 1025, 2048, 2049, 32768, 65537, 131072, 200000, 1 << 20, (1 << 28) - 1, 1 << 28):
            for drawn, children in ((0, 1), (1, 1), (1, 2), (0, 9)):
                host.kvt_verify_plan(batch, vocab, drawn, children, cus, out)
                parts, part, rounds = out
                assert 1 <= parts <= 64 and part % 1024 == 0 and (parts - 1) * part < vocab <= parts * part
                assert rounds == (1 if drawn and children > 1 else 0)
                assert batch * parts * 256 <= 1 << 31
                need = batch * (parts * 32 + 128)
                for more in ((batch, vocab), (batch + 1, vocab), (min(2 * batch, 1 << 20), min(1 << 28, 3 * vocab)), (1 << 20, 1 << 28)):
                    assert need <= host.kvt_verify_bound(*more, cus)


PLAN = ("rows", "many", "tiles", "items", "slots", "places", "least", "most_runs", "partials", "join_rows", "join_groups",
        "join_grid", "ws_bytes")


def _plan(host, *shape):
    out = (ctypes.c_int64 * len(PLAN))()
    host.kvt_plan(*shape, out)
    return dict(zip(PLAN, out))


HEADS = [(64, 8), (96, 8), (8, 8), (1, 1), (1024, 1), (1024, 1024), (12, 4)]


@pytest.mark.parametrize("cus", [32, 256, 304])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_plans_hold_any_lengths(host, D, cus):
    """What the kernels make of a batch's lengths - those of the bounds, shorter and longer ones - fits the grid, the
    partials and the list of items to join."""
    r = np.random.default_rng(D + cus)
    for _ in range(1500):
        Hq, Hkv = HEADS[r.integers(len(HEADS))]
        batch, max_q, max_kv = (int(np.exp(r.uniform(0, np.log(top)))) for top in (600, 1100, 1 << 22))
        f32 = int(r.integers(2))
        p = _plan(host, Hq, Hkv, D, batch, max_q, max_kv, f32, cus)
        assert p["items"] == batch * Hkv * p["tiles"] and p["tiles"] * p["rows"] >= max_q * Hq // Hkv
        assert p["items"] >= 1 << 23 or p["slots"] * 512 < 1 << 32
        assert p["rows"] in {64: (16, 32, 64, 128), 128: (16, 32, 128, 256) if f32 else (16, 32, 64, 128, 256), 256: (16, 32, 128)}[D]
        if p["slots"] == p["items"]:
            assert p["ws_bytes"] == 0 or batch > 512
            continue
        assert p["ws_bytes"] == p["partials"] * p["rows"] * (D + 2) * 4 + 16 + 32 * min(p["items"], p["places"])
        assert (p["join_rows"] or 1) * p["join_groups"] >= min(p["rows"], max_q * Hq // Hkv)
        for top in (max_kv, 1 << 12, (1 << 31) - 1, max(1, max_kv // 50)):
            n = min(batch, 512)
            lens = np.minimum(top, np.exp(r.uniform(0, np.log(top + 1), n))).astype(np.int64)
            if r.random() < 0.4:
                lens[:] = top
            blocks = np.ascontiguousarray(-(-lens // 32), dtype=np.int32)
            queries = np.ascontiguousarray(r.integers(0, max_q + 1, n) if r.random() < 0.5 else np.full(n, max_q), dtype=np.int32)
            at = lambda x: x.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))  # noqa: E731
            got = [ctypes.c_int64() for _ in range(3)]
            chunk = host.kvt_shared(Hkv, n, at(blocks), at(queries), *[ctypes.byref(x) for x in got])
            work, partials, joins = (x.value for x in got)
            assert work <= p["slots"] and partials <= p["partials"] and joins <= min(p["items"], p["places"])
            assert -(-int(blocks.max()) // chunk) <= 256


@pytest.mark.parametrize("cus", [32, 256, 304])
def test_tree_workspace_of_bounds_holds_every_smaller_call(host, cus):
    r = np.random.default_rng(cus)
    for _ in range(4000):
        Hq, Hkv = HEADS[r.integers(len(HEADS))]
        D = (64, 128, 256)[r.integers(3)]
        most = [int(np.exp(r.uniform(0, np.log(top)))) for top in (2000, 1100, 1 << 20)]
        less = [int(np.exp(r.uniform(0, np.log(top)))) for top in most]
        bound = host.kvt_bound(Hq, Hkv, D, *most, cus)
        for f32 in (0, 1):
            assert _plan(host, Hq, Hkv, D, *less, f32, cus)["ws_bytes"] <= bound
            assert _plan(host, Hq, Hkv, D, *most, f32, cus)["ws_bytes"] <= bound


def test_gpu_tests_reach_every_form(host):
    from tests import test_gpu_kv_tree as t
    seen = set()
    for Hq, Hkv, D, page, shape, max_kv in t.FORMS:
        width = max(1, max(-(-n // page) for _, n in shape)) * page
        for f32 in (0, 1):
            p = _plan(host, Hq, Hkv, D, len(shape), max(n for n, _ in shape), max_kv or width, f32, 256)
            seen.add((D, p["rows"], p["slots"] > p["items"], p["join_rows"] > 0 if p["slots"] > p["items"] else None))
    several = {(D, n, True) for D, rows in ((64, (16, 32, 64, 128)), (128, (16, 32, 64, 128, 256)), (256, (16, 32, 128))) for n in rows}
    one = {(D, n, False) for D, n, _ in several} - {(128, 32, False)}
    assert {x[:3] for x in seen} >= one | several - {(128, 128, True)}  # one run of 32, several of 128: only larger calls
    assert {x[3] for x in seen} == {None, False, True}


def test_tree_plans_at_the_ends(host):
    assert _plan(host, 64, 8, 128, 0, 5, 100, 0, 256)["items"] == 0
    p = _plan(host, 64, 8, 128, 1, 1, 1 << 40, 0, 256)
    assert p["partials"] <= 1024 and p["most_runs"] == 256
    assert _plan(host, 1024, 1, 64, 1 << 20, 1024, 1 << 31, 1, 256)["items"] >= 1 << 23  # refused for its items
    for max_q in (1 << 13, 1 << 16, 1 << 18, 1 << 20, 1 << 23):  # many items: one run each, in a grid that can be launched
        for shape in ((1024, 1), (64, 8), (8, 8)):
            p = _plan(host, *shape, 128, 512, max_q, 1 << 20, 0, 256)
            assert p["items"] >= 1 << 23 or p["slots"] * 512 < 1 << 32


def test_reports(host):
    text = ctypes.create_string_buffer(256)

    def say(*a):
        host.kvt_report(*a, text)
        return text.value.decode()
    assert say(7, 5, -9) == "row 5: parent -9 is no earlier node of its tree"
    assert say(8, 8388607, 1 << 40) == "row 8388607: drafted token from 34359738367 outside the vocabulary"
    assert say(9, 3, 0) == "sequence 3: no probability to draw from"
    assert say(10, 0, -2) == "sequence 0: a path of -2 nodes that does not ascend within its tree"


# ---------------------------------------------------------------- oracle

def test_masks_and_visibility():
    parent = [-1, 0, 0, 1, 3, 2, -1]
    assert okt.ancestors(parent) == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 1, 3, 4}, {0, 2, 5}, {6}]
    m = okt.masks([-1] + list(range(70)), 2)
    assert m[70].tolist() == [2 ** 64 - 1, 127] and m[63].tolist() == [2 ** 64 - 1, 0]
    m = okt.masks(parent, 1)
    want = [[True] * 3 + [j in s for j in range(7)] for s in okt.ancestors(parent)]
    np.testing.assert_array_equal(okt.visible(m, 3, 10), want)
    np.testing.assert_array_equal(okt.visible(m, 3, 5), np.array(want)[:, :5])
    np.testing.assert_array_equal(okt.visible(m, -2, 5), np.array(want)[:, 5:])
    assert not okt.visible(m, -100, 20).any()


def test_attend_agrees_with_the_causal_oracle_on_a_chain():
    from oracle import kv as okv
    r = np.random.default_rng(3)
    q, K, V = r.standard_normal((5, 4, 64)), r.standard_normal((12, 2, 64)), r.standard_normal((12, 2, 64))
    m = okt.masks([-1, 0, 1, 2, 3], 1)
    for a, b in zip(okt.attend(q, K, V, okt.visible(m, 7, 12), 0.1), okv.attend(q, K, V, [8, 9, 10, 11, 12], 0.1)):
        # sums of 64 and of 12 terms, below 8 in size, in two orders: an entry that cancels is off by 76 * 8 * 2^-53 at most
        np.testing.assert_allclose(a, b, rtol=1e-13, atol=76 * 8 * 2.0 ** -53)


def _grid(n):
    return (np.arange(n) + 0.5) / n


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_verified_tokens_are_the_targets_drawn(kids):
    """Over all drafts without replacement, with their chances, and a grid of the random numbers the first token that
    comes out has the target's distribution, to the grid's step."""
    p, q = np.array([[0.5, 0.05, 0.15, 0.3]]), np.array([[0.1, 0.6, 0.25, 0.05]])
    steps = {1: 60, 2: 16, 3: 8}[kids]
    rows = np.repeat(p, kids + 1, 0), np.repeat(q, kids + 1, 0)
    got = np.zeros(4)
    for drafts in itertools.permutations(range(4), kids):
        chance, left = 1.0, 1.0
        for x in drafts:
            chance *= q[0, x] / left
            left -= q[0, x]
        for u in itertools.product(_grid(steps), repeat=kids + 1):
            path, nxt, _ = okt.verify((0,) + drafts, [-1] + [0] * kids, *rows, u)
            got[drafts[path[1] - 1] if len(path) > 1 else nxt] += chance / steps ** (kids + 1)
    # each of the kids + 1 numbers' intervals is off by half a step at either end
    np.testing.assert_allclose(got, p[0], atol=(kids + 1) / steps)
    assert abs(got - p[0]).sum() < (kids + 1) / steps


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_verified_tokens_are_the_targets_certain(kids):
    p, steps = np.array([0.5, 0.05, 0.15, 0.3]), {1: 60, 2: 20, 3: 8}[kids]
    got = np.zeros(4)
    drafts = (2, 0, 3)[:kids]
    for u in itertools.product(_grid(steps), repeat=kids + 1):
        path, nxt, _ = okt.verify((0,) + drafts, [-1] + [0] * kids, np.repeat(p[None], kids + 1, 0), None, u)
        got[drafts[path[1] - 1] if len(path) > 1 else nxt] += 1 / steps ** (kids + 1)
    np.testing.assert_allclose(got, p, atol=(kids + 1) / steps)


def test_verify_walks_down_and_passes_over_what_it_cannot_use():
    p = np.full((6, 4), 0.25)
    #            root 0 -> 1 (token 2), 2 (token 2 again), 3 (outside), 4 (token 1); 4 -> 5
    token, parent = [0, 2, 2, 9, 1, 3], [-1, 0, 0, 0, 0, 4]
    assert okt.verify(token, parent, p, None, [0.1, 0.3, 0.0, 0.0, 0.3, 0.2])[:2] == ([0, 4, 5], 0)
    assert okt.verify(token, parent, p, None, [0.1, 0.2, 0.0, 0.0, 0.0, 0.0])[:2] == ([0, 1], 0)
    assert okt.verify(token, parent, p, None, [0.6, 0.9, 0.0, 0.0, 0.9, 0.0])[:2] == ([0], 3)  # tokens 0 and 3 are left
    assert okt.verify([0], [-1], np.zeros((1, 4)), None, [0.5])[:2] == ([0], -1)
    # ties: a number on the border is not below it
    assert okt.verify(token, parent, p, None, [0.5, 0.25, 0, 0, 0.25, 0.25])[:2] == ([0, 4], 1)  # 0.375 of 0, 1, 2
    assert okt.verify([0], [-1], p[:1], None, [0.25])[:2] == ([0], 1)
