"""The key/value cache on the CPU (no GPU): its oracle, its page layout and its refusals.

tests/kv_host_check.cpp compiles the host library's own argument checks and
the kernels' own layout functions (csrc/kv_checks.h, csrc/kv_layout.h) with
g++, so that every refusal is tested before anything could be launched.
"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import kv as okv
from shard_decomposed_gemm_amd import agemm, kvc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kvcache.h")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    so = str(tmp_path_factory.mktemp("kvh") / "kvh.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "shard_decomposed_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "kv_host_check.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    shape = [ctypes.c_int] * 4 + [i64]
    lib.kvh_create.argtypes = shape
    lib.kvh_append.argtypes = shape + [vp, ctypes.POINTER(kvc.AppendArgs), ctypes.c_char_p]
    lib.kvh_attend.argtypes = shape + [vp, ctypes.POINTER(kvc.AttendArgs), i64, vp, i64, ctypes.c_char_p]
    lib.kvh_read.argtypes = [vp, i64, vp, vp, vp, ctypes.c_char_p]
    lib.kvh_block.argtypes = shape + [i64, ctypes.c_int] + [ctypes.POINTER(ctypes.c_int)] * 3
    lib.kvh_block.restype = i64
    lib.kvh_plan.argtypes = shape + [i64, i64, i64, ctypes.c_int, ctypes.POINTER(i64)]
    lib.kvh_plan.restype = None
    lib.kvh_chunk.argtypes = [i64, ctypes.c_int]
    lib.kvh_many_items.argtypes = [ctypes.c_int] * 3 + [i64] * 4 + [ctypes.c_int] + [ctypes.POINTER(i64)] * 2
    lib.kvh_many_items.restype = i64
    return lib


# ---------------------------------------------------------------- interface

def test_header_matches_binding():
    import re
    names = sorted(set(re.findall(r"^\s*(?:int|const char\*)\s+(kvc_[a-z_]+)\s*\(", open(HEADER).read(), re.M)))
    assert sorted(kvc.EXPORTED) == names
    lib = kvc.load()
    for name in names:
        assert hasattr(lib, name), name


def test_argument_structs_have_the_headers_size(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src = tmp_path / "s.c"
    fields = {"kvc_append_args": kvc.AppendArgs, "kvc_attend_args": kvc.AttendArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kvcache.h"', "int main(void) {"]
    for name, st in fields.items():
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        lines += [f'  printf("%zu\\n", offsetof({name}, {f[0]}));' for f in st._fields_]
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    exe = str(tmp_path / "s")
    subprocess.run([gxx, "-x", "c", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    want = []
    for st in fields.values():
        want += [ctypes.sizeof(st)] + [getattr(st, f[0]).offset for f in st._fields_]
    assert [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()] == want


def test_packed_arguments_are_the_structs():
    for st, pack in ((kvc.AppendArgs, kvc._pack_append), (kvc.AttendArgs, kvc._pack_attend)):
        values = [i + 1 if t is not ctypes.c_float else i + 0.5 for i, (_, t) in enumerate(st._fields_)]
        assert len(pack(*values)) <= ctypes.sizeof(st)  # without the padding at the end
        got = st.from_buffer_copy(pack(*values).ljust(ctypes.sizeof(st), b"\0"))
        assert [getattr(got, name) for name, _ in st._fields_] == values


# ---------------------------------------------------------------- oracle

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page_tokens", [32, 64, 256])
def test_pack_and_unpack_are_inverse_and_fill_every_byte(D, page_tokens):
    r = np.random.default_rng(D + page_tokens)
    S, H = 2 * page_tokens, 3
    n = lambda: r.integers(0, 16, (S, H, D), dtype=np.uint8)  # noqa: E731
    p = lambda: r.standard_normal((S, H, 1)).astype(np.float16)  # noqa: E731
    parts = (n(), p(), p(), n(), p(), p())
    pages = okv.pack(*parts, page_tokens)
    assert pages.shape == (2, H * page_tokens * (D + 8))
    for got, want in zip(okv.unpack(pages, H, D, page_tokens), parts):
        np.testing.assert_array_equal(got, want)
    # as many bits as numbers: random bytes survive the way there and back too
    raw = r.integers(0, 256, pages.shape, dtype=np.uint8)
    np.testing.assert_array_equal(okv.pack(*okv.unpack(raw, H, D, page_tokens), page_tokens), raw)


def test_quantised_values_are_within_half_a_step():
    r = np.random.default_rng(5)
    x = r.standard_normal((200, 4, 128)) * np.exp(3 * r.standard_normal((200, 4, 1)))
    n, s, b, _ = okv.quantise(x)
    v = okv.held(n, s, b)
    s, b = s.astype(np.float64), b.astype(np.float64)
    x = np.clip(x, -okv.LIMIT, okv.LIMIT)
    # Half a step; at the ends the 15 steps of s and b are off by half a unit in the last place each (2^-11 of the
    # number, 2^-25 where it is subnormal), and the held value, |v| <= |x| + s, is rounded to binary16.
    half = lambda y: np.maximum(np.abs(y) * 2.0 ** -11, 2.0 ** -25)  # noqa: E731
    bound = s / 2 + 15 * half(s) + half(b) + half(np.abs(x) + s)
    assert (np.abs(v - x) <= bound).all()


def test_quantise_constant_zero_and_nonfinite_rows():
    n, s, b, _ = okv.quantise(np.full((1, 64), 0.75))
    assert (n == 0).all() and s == 0 and b == np.float16(0.75)
    assert (okv.held(n, s, b) == 0.75).all()
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 2] = np.inf, -np.inf, np.nan
    n, s, b, _ = okv.quantise(x)
    v = okv.held(n, s, b)
    assert np.isfinite(v).all() and abs(v[0, 0] - okv.LIMIT) < 32 and abs(v[0, 1] + okv.LIMIT) < 32


def test_attend_oracle_against_a_direct_product():
    r = np.random.default_rng(7)
    q, K, V = r.standard_normal((3, 4, 64)), r.standard_normal((9, 2, 64)), r.standard_normal((9, 2, 64))
    O, lse, _, _ = okv.attend(q, K, V, [0, 5, 9], 0.125)
    assert (O[0] == 0).all() and (lse[0] == okv.LOWEST).all()
    for i, L in ((1, 5), (2, 9)):
        for h in range(4):
            w = np.exp(0.125 * K[:L, h // 2] @ q[i, h])
            np.testing.assert_allclose(O[i, h], (w[:, None] * V[:L, h // 2]).sum(0) / w.sum(), rtol=1e-12)
            np.testing.assert_allclose(lse[i, h], np.log(w.sum()), rtol=1e-12)


# ---------------------------------------------------------------- layout

@pytest.mark.parametrize("D,page_tokens,Hkv", [(64, 32, 3), (128, 64, 2), (256, 256, 1)])
def test_layout_functions_agree_with_the_oracle(host, D, page_tokens, Hkv):
    num_pages = 1 << 33  # offsets beyond 32 bits
    c = [ctypes.c_int() for _ in range(3)]
    page_bytes = Hkv * page_tokens * (D + 8)
    _, _, _, (at, _) = okv._places(D)
    for page in (0, 7, num_pages // page_tokens - 1):
        for off in (0, 1, 5, 31, page_tokens // 2, page_tokens - 1):
            for h in range(Hkv):
                got = host.kvh_block(Hkv, Hkv, D, page_tokens, num_pages, page * page_tokens + off, h,
                                     *[ctypes.byref(x) for x in c])
                assert got == page * page_bytes + (h * (page_tokens // 32) + off // 32) * 32 * (D + 8)
                assert c[0].value == off % 32
                assert 32 * D + 128 + 2 * (8 * c[1].value + c[2].value) == at[off % 32]


@pytest.mark.parametrize("Hq,Hkv,D", [(64, 8, 128), (96, 96, 128), (12, 1, 128), (16, 2, 256), (32, 4, 64), (72, 1, 64)])
def test_plan_covers_every_block_once_within_its_workspace(host, Hq, Hkv, D):
    """Runs of blocks partition every length, the longest that fits 32 bits among them, in no more runs than the grid,
    the workspace and the join have; longer sequences than max_kv are covered too."""
    v = (ctypes.c_int64 * 11)()
    r = np.random.default_rng(Hq)
    for batch in (1, 2, 7, 64, 500, 8192):
        for max_q in (1, 2, 5, 33, 700):
            for max_kv in (1, 33, 777, 4099, 65536, 262144, (1 << 31) - 1):
                host.kvh_plan(Hq, Hkv, D, 64, 1000, batch, max_q, max_kv, 256, v)
                many, rows, join_rows, join_groups, tiles, splits, chunk, items, slots, slot, ws = v
                live = min(rows, max_q * (Hq // Hkv))
                assert items == batch * Hkv * tiles and slot == rows * (D + 2)
                assert tiles * rows >= max_q * (Hq // Hkv) and (many or tiles == 1)
                assert join_rows * join_groups >= live and join_rows in (1, 2048 // D)
                top = min((max_kv + 31) // 32, 1 << 26)
                if many:
                    assert 1 <= splits <= 256 and chunk >= 1
                    assert ws == (items * splits * slot * 4 if splits > 1 else 0)
                    assert splits == 1 or items < 1 << 24  # the join's grid
                    for n in (0, 1, 2, 31, 32, 33, 64, 1000, top, min(3 * top, 1 << 26), 1 << 26):
                        c, k = host.kvh_run_blocks(chunk, splits, n), host.kvh_runs(chunk, splits, n)
                        assert 1 <= k <= splits and c >= 1
                        assert (k - 1) * c < max(n, 1) <= k * c < 1 << 31
                        assert n > 0 or k == 1
                    for T in (max_q, 1, batch * max_q, batch + max_q):
                        wide, wtiles = ctypes.c_int64(), ctypes.c_int64()
                        grid = host.kvh_many_items(Hq, Hkv, D, batch, max_q, max_kv, T, 256, wide, wtiles)
                        wide, wtiles = wide.value, wtiles.value
                        assert wide == rows or (wide == 256 and splits == 1 and grid >= 1024)
                        assert wide * wtiles >= max_q * (Hq // Hkv) and 0 < grid <= batch * wtiles * Hkv
                        # T rows cut into sequences of max_q at most, in whatever way
                        cuts = np.sort(r.integers(0, T + 1, batch - 1)) if batch > 1 else np.empty(0, np.int64)
                        n = np.minimum(np.diff(np.concatenate([[0], cuts, [T]])), max_q)
                        assert (-(-n * (Hq // Hkv) // wide)).sum() * Hkv <= grid
                    continue
                assert splits == 1 and slots < 1 << 23
                assert ws == (slots * slot * 4 if slots > items else 0)
                for kind in range(4):
                    n = np.minimum(np.maximum(0, [np.full(batch, top), np.full(batch, 3 * top),
                                                  (top ** r.random(batch)).astype(np.int64),
                                                  np.where(np.arange(batch) == 0, 1 << 26, r.integers(0, 3, batch))][kind]), 1 << 26)
                    c = host.kvh_chunk(int(n.sum()) * Hkv, int(n.max()))
                    runs = np.maximum(1, -(-n // c))
                    assert runs.sum() * Hkv <= slots and (slots == items or runs.max() <= 256)
                    assert [host.kvh_item_runs(c, int(x)) for x in n[:20]] == runs[:20].tolist()
                    assert c <= 1 << 26 and int(runs.max()) * c < 1 << 31


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (64, 8), (96, 96), (1024, 1), (1024, 1024), (1023, 1023), (5, 5)])
def test_launches_of_append_and_read_stay_within_32_bits(host, Hq, Hkv):
    host.kvh_piece.restype = ctypes.c_int64
    for D in (64, 128, 256):
        quads = max(-(-Hq // 4), 2 * -(-Hkv // 4))
        rows = host.kvh_piece(Hq, Hkv, D, 0) * quads
        # four quads a wave, four waves a workgroup of 256 threads; the read: 16 threads a row
        assert 0 < rows < 1 << 28 and -(-rows // 16) * 256 < 1 << 32
        assert 0 < -(-host.kvh_piece(Hq, Hkv, D, 1) * Hkv // 16) * 256 < 1 << 32


# ---------------------------------------------------------------- refusals

SHAPE = (16, 4, 128, 64, 10)


@pytest.mark.parametrize("shape", [
    (16, 0, 128, 64, 10), (4, 16, 128, 64, 10), (16, 5, 128, 64, 10), (2048, 4, 128, 64, 10), (16, 4, 96, 64, 10),
    (16, 4, 128, 16, 10), (16, 4, 128, 96, 10), (16, 4, 128, 512, 10), (16, 4, 128, 64, 0),
    (16, 4, 128, 64, (1 << 40) // 64 + 1), (0, 0, 128, 64, 1)])
def test_create_refuses_shapes(host, shape):
    assert host.kvh_create(*shape) == agemm.ESHAPE
    h = ctypes.c_void_p()
    assert kvc.load().kvc_create(ctypes.byref(h), *shape) == agemm.ESHAPE and not h.value
    assert host.kvh_create(*SHAPE) == agemm.OK


def _append(**change):
    base = dict(tokens=5, q=0x1000, k=0x2000, v=0x3000, q_out=0x4000, q_token_stride=2048, q_head_stride=128,
                k_token_stride=512, k_head_stride=128, v_token_stride=512, v_head_stride=128, out_token_stride=2048,
                out_head_stride=128, slots=0x5000, positions=0x6000, rope=0x7000, rope_len=100, rope_dims=128,
                interleaved=0, q_norm=0x8000, k_norm=0x9000, eps=1e-6)
    assert set(change) <= set(base) and len(base) == len(kvc.AppendArgs._fields_)
    return kvc.AppendArgs(**{**base, **change})


def test_append_accepts(host):
    why = ctypes.create_string_buffer(256)
    ok = lambda pages=0x10000, **c: host.kvh_append(*SHAPE, pages, _append(**c), why)  # noqa: E731
    assert ok() == agemm.OK
    assert ok(rope=None, positions=None, rope_dims=0, rope_len=0) == agemm.OK
    assert ok(q_norm=None, k_norm=None, eps=float("nan")) == agemm.OK  # eps unused
    assert ok(pages=None, k=None, v=None, k_norm=None, slots=None) == agemm.OK  # queries alone
    assert ok(q=None, q_out=None, q_norm=None, q_token_stride=3) == agemm.OK  # keys and values alone
    assert ok(q_out=0x1000) == agemm.OK  # in place
    assert ok(out_token_stride=128, out_head_stride=640) == agemm.OK  # heads outside
    assert ok(k_token_stride=0, q_head_stride=0) == agemm.OK  # broadcast inputs
    assert ok(slots=0x5008, positions=0x6018, rope=0x7004) == agemm.OK  # index slices
    assert ok(tokens=0, q=None, k=None, v=None, q_out=None) == -1  # nothing to do


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), agemm.EINVAL), (dict(tokens=(1 << 23) + 1), agemm.ESHAPE),
    (dict(q=None, k=None, v=None), agemm.EINVAL), (dict(v=None), agemm.EINVAL), (dict(k=None), agemm.EINVAL),
    (dict(q_out=None), agemm.EINVAL), (dict(q=None), agemm.EINVAL), (dict(q=None, q_out=None), agemm.EINVAL),
    (dict(slots=None), agemm.EINVAL), (dict(positions=None), agemm.EINVAL),
    (dict(rope_dims=0), agemm.EINVAL), (dict(rope_dims=24), agemm.EINVAL), (dict(rope_dims=144), agemm.EINVAL),
    (dict(rope_len=0), agemm.EINVAL), (dict(interleaved=2), agemm.EINVAL), (dict(eps=-1.0), agemm.EINVAL),
    (dict(eps=float("nan")), agemm.EINVAL), (dict(eps=float("inf")), agemm.EINVAL),
    (dict(q=0x1008), agemm.EINVAL), (dict(k=0x2004), agemm.EINVAL), (dict(v=0x3002), agemm.EINVAL),
    (dict(q_out=0x4008), agemm.EINVAL), (dict(q_norm=0x8002), agemm.EINVAL), (dict(k_norm=0x9008), agemm.EINVAL),
    (dict(slots=0x5004), agemm.EINVAL), (dict(positions=0x6004), agemm.EINVAL), (dict(rope=0x7002), agemm.EINVAL),
    (dict(q_token_stride=2052), agemm.EINVAL), (dict(q_head_stride=-128), agemm.EINVAL),
    (dict(k_token_stride=516), agemm.EINVAL), (dict(v_head_stride=-8), agemm.EINVAL),
    (dict(v_token_stride=1 << 41), agemm.EINVAL),
    (dict(out_head_stride=64), agemm.EINVAL), (dict(out_token_stride=0), agemm.EINVAL),
    (dict(out_token_stride=1024), agemm.EINVAL),
    (dict(q_out=0x1000, out_token_stride=4096), agemm.EINVAL),
])
def test_append_refuses(host, change, code):
    why = ctypes.create_string_buffer(256)
    assert host.kvh_append(*SHAPE, 0x10000, _append(**change), why) == code
    assert why.value


def test_append_refuses_pages_and_null(host):
    why = ctypes.create_string_buffer(256)
    for pages in (None, 0x10008):
        assert host.kvh_append(*SHAPE, pages, _append(), why) == agemm.EINVAL
    assert host.kvh_append(*SHAPE, 0x10000, None, why) == agemm.EINVAL


def _attend(**change):
    base = dict(batch=3, max_q=4, tokens=12, q=0x1000, q_token_stride=2048, q_head_stride=128, q_start=0x2000,
                kv_len=0x3000, q_off=0x4000, page_table=0x5000, table_stride=8, table_width=8, causal=1, max_kv=512,
                scale=0.1, out_f32=1, out=0x6000, lse=0x7000)
    assert set(change) <= set(base) and len(base) == len(kvc.AttendArgs._fields_)
    return kvc.AttendArgs(**{**base, **change})


def test_attend_accepts(host):
    why = ctypes.create_string_buffer(256)
    ok = lambda need=0, ws=None, n=0, **c: host.kvh_attend(*SHAPE, 0x10000, _attend(**c), need, ws, n, why)  # noqa: E731
    assert ok() == agemm.OK
    assert ok(lse=None, q_off=None, out_f32=0, causal=0) == agemm.OK
    assert ok(q_start=None, max_q=1) == agemm.OK
    assert ok(table_stride=0) == agemm.OK
    assert ok(kv_len=0x3004, lse=0x7004, q_start=0x2008, page_table=0x500c) == agemm.OK
    assert ok(need=64, ws=0x8000, n=64) == agemm.OK
    assert ok(batch=0, q=None, kv_len=None, page_table=None, out=None) == -1
    assert ok(tokens=0, q=None, out=None) == -1


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), agemm.EINVAL), (dict(tokens=-1), agemm.EINVAL), (dict(max_q=0), agemm.EINVAL),
    (dict(max_kv=0), agemm.EINVAL), (dict(tokens=(1 << 23) + 1), agemm.ESHAPE), (dict(max_q=(1 << 23) + 1), agemm.ESHAPE),
    (dict(batch=(1 << 23) + 1), agemm.ESHAPE), (dict(batch=1 << 22, max_q=1 << 8), agemm.ESHAPE), (dict(causal=2), agemm.EINVAL), (dict(out_f32=2), agemm.EINVAL),
    (dict(scale=float("nan")), agemm.EINVAL), (dict(scale=float("inf")), agemm.EINVAL),
    (dict(table_width=0), agemm.EINVAL), (dict(table_stride=7), agemm.EINVAL), (dict(table_stride=-8), agemm.EINVAL),
    (dict(q_start=None), agemm.EINVAL), (dict(q_start=None, max_q=1, batch=13), agemm.EINVAL),
    (dict(q_token_stride=2050), agemm.EINVAL), (dict(q_head_stride=-8), agemm.EINVAL),
    (dict(q=None), agemm.EINVAL), (dict(q=0x1008), agemm.EINVAL), (dict(out=None), agemm.EINVAL),
    (dict(out=0x6004), agemm.EINVAL), (dict(kv_len=None), agemm.EINVAL), (dict(page_table=None), agemm.EINVAL),
    (dict(kv_len=0x3002), agemm.EINVAL), (dict(page_table=0x5001), agemm.EINVAL), (dict(q_off=0x4002), agemm.EINVAL),
    (dict(q_start=0x2002), agemm.EINVAL), (dict(lse=0x7002), agemm.EINVAL),
])
def test_attend_refuses(host, change, code):
    why = ctypes.create_string_buffer(256)
    assert host.kvh_attend(*SHAPE, 0x10000, _attend(**change), 0, None, 0, why) == code
    assert why.value


def test_attend_refuses_pages_workspace_and_null(host):
    why = ctypes.create_string_buffer(256)
    for pages in (None, 0x10004):
        assert host.kvh_attend(*SHAPE, pages, _attend(), 0, None, 0, why) == agemm.EINVAL
    for ws, n in ((None, 64), (0x8000, 63), (0x8008, 64)):
        assert host.kvh_attend(*SHAPE, 0x10000, _attend(), 64, ws, n, why) == agemm.EINVAL
    assert host.kvh_attend(*SHAPE, 0x10000, None, 0, None, 0, why) == agemm.EINVAL


@pytest.mark.parametrize("args,code", [
    ((0x1000, 4, 0x2000, 0x3000, 0x4000), agemm.OK), ((0x1000, 4, 0x2008, 0x3000, 0x4000), agemm.OK),
    ((0x1000, 0, None, None, None), -1), ((0x1000, -1, 0x2000, 0x3000, 0x4000), agemm.EINVAL),
    ((0x1000, (1 << 23) + 1, 0x2000, 0x3000, 0x4000), agemm.ESHAPE), ((None, 4, 0x2000, 0x3000, 0x4000), agemm.EINVAL),
    ((0x1008, 4, 0x2000, 0x3000, 0x4000), agemm.EINVAL), ((0x1000, 4, None, 0x3000, 0x4000), agemm.EINVAL),
    ((0x1000, 4, 0x2004, 0x3000, 0x4000), agemm.EINVAL), ((0x1000, 4, 0x2000, None, 0x4000), agemm.EINVAL),
    ((0x1000, 4, 0x2000, 0x3008, 0x4000), agemm.EINVAL), ((0x1000, 4, 0x2000, 0x3000, 0x4008), agemm.EINVAL),
])
def test_read_refuses(host, args, code):
    assert host.kvh_read(*args, ctypes.create_string_buffer(256)) == code


def test_calls_without_a_context_are_refused():
    lib = kvc.load()
    n = ctypes.c_int64()
    assert lib.kvc_append(None, None, ctypes.byref(_append()), None) == agemm.EINVAL
    assert lib.kvc_attend(None, None, ctypes.byref(_attend()), None, 0, None) == agemm.EINVAL
    assert lib.kvc_read(None, None, 0, None, None, None, None) == agemm.EINVAL
    assert lib.kvc_check(None) == agemm.EINVAL
    assert lib.kvc_page_bytes(None, ctypes.byref(n)) == agemm.EINVAL
    assert lib.kvc_attend_workspace(None, 1, 1, 1, ctypes.byref(n)) == agemm.EINVAL
    assert lib.kvc_destroy(None) == agemm.OK
    assert lib.kvc_last_error(None) == b""
