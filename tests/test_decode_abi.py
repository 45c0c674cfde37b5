"""The decode operators' C ABI (CPU): symbols, struct layouts, and the refusals that come
before any CUDA call."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from bucketized_guidance_step_gb300 import build, decode, gs

HEADER = os.path.join(build.INCLUDE, "gs_decode.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return decode.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(HEADER).read()
    names = re.findall(r"^\s*gs_status\s+(gs_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(decode.EXPORTS)
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


def test_constants_match_the_header():
    text = open(HEADER).read()
    for name in ("GS_DEV_NO_PAGE", "GS_DEV_BAD_SEQ", "GS_DEV_EMPTY_ROW", "GS_MAX_SEQS"):
        assert int(re.search(rf"#define {name}\s+(\d+)", text).group(1)) == getattr(decode, name)


def test_ctypes_structs_match_the_header_layout(lib, repo_tmp):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = {"gs_kv_cache": decode.KVCacheDesc, "gs_paged_attention_args": decode.PagedAttentionArgs,
             "gs_guided_logits_args": decode.GuidedLogitsArgs}
    lines = [f'printf("{c} sizeof %zu\\n", sizeof({c}));' for c in pairs]
    lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for c, py in pairs.items() for f, _ in py._fields_]
    src = repo_tmp / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"gs_decode.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = repo_tmp / "layout"
    subprocess.run([cc, "-std=c11", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        s, m, v = line.split()
        got[s, m] = int(v)
    for c, py in pairs.items():
        assert got[c, "sizeof"] == ctypes.sizeof(py), c
        for f, _ in py._fields_:
            assert got[c, f] == getattr(py, f).offset, (c, f)


def test_status_words(lib):
    assert decode.status_from_word(0) == gs.GS_OK
    assert decode.status_from_word(decode.GS_DEV_NO_PAGE) == gs.GS_ERR_CAPACITY
    assert decode.status_from_word(decode.GS_DEV_BAD_SEQ) == gs.GS_ERR_INVALID_ARG
    assert decode.status_from_word(decode.GS_DEV_EMPTY_ROW) == gs.GS_ERR_UNSUPPORTED
    assert decode.status_from_word(gs.GS_DEV_STEP_RANGE) == gs.GS_ERR_STEP_RANGE


def _cache():
    d = decode.KVCacheDesc()
    d.dtype, d.layers, d.pages, d.kv_heads, d.page, d.dim = gs.GS_DTYPE_BF16, 2, 8, 2, 16, 64
    d.token_stride, d.head_stride, d.page_stride, d.layer_stride = 64, 1024, 2048, 16384
    d.k = d.v = 0x10000
    d.seqs, d.cols = 4, 4
    d.table, d.lens, d.refs = 0x20000, 0x30000, 0x40000
    d.workspace, d.workspace_bytes = 0x50000, 1 << 20
    return d


CACHE_REFUSALS = [
    ("dtype", 7, gs.GS_ERR_INVALID_ARG), ("layers", 0, gs.GS_ERR_INVALID_ARG),
    ("pages", 0, gs.GS_ERR_INVALID_ARG), ("kv_heads", -1, gs.GS_ERR_INVALID_ARG),
    ("page", 0, gs.GS_ERR_INVALID_ARG), ("dim", 0, gs.GS_ERR_INVALID_ARG),
    ("dim", 60, gs.GS_ERR_UNSUPPORTED), ("dim", 264, gs.GS_ERR_UNSUPPORTED),
    ("k", None, gs.GS_ERR_INVALID_ARG), ("v", 0x10008, gs.GS_ERR_UNSUPPORTED),
    ("table", None, gs.GS_ERR_INVALID_ARG), ("lens", None, gs.GS_ERR_INVALID_ARG),
    ("refs", None, gs.GS_ERR_INVALID_ARG), ("lens", 0x30002, gs.GS_ERR_INVALID_ARG),
    ("token_stride", 68, gs.GS_ERR_UNSUPPORTED), ("head_stride", -64, gs.GS_ERR_INVALID_ARG),
    ("token_stride", 32, gs.GS_ERR_INVALID_ARG), ("seqs", 0, gs.GS_ERR_INVALID_ARG),
    ("seqs", 8193, gs.GS_ERR_UNSUPPORTED), ("cols", 1 << 28, gs.GS_ERR_UNSUPPORTED),
    ("cols", (1 << 26) + 1, gs.GS_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("field,value,status", CACHE_REFUSALS)
def test_cache_refusals(lib, field, value, status):
    d = _cache()
    setattr(d, field, value)
    r = ctypes.byref(d)
    assert lib.gs_pages_extend(r, 0x60000, None, 1, None) == status
    assert lib.gs_pages_fork(r, 0x60000, 0x60010, 1, None) == status
    assert lib.gs_pages_free(r, 0x60000, 1, None) == status
    assert lib.gs_pages_compact(r, 0x60000, 0x60000, None, None) == status
    assert lib.gs_kv_write(r, 0, 0x60000, 0x60000, 128, 64, 1, 0x60000, 0x60000, 1, None) == status
    a = _attention(d)
    assert lib.gs_paged_attention(ctypes.byref(a), None) == status


def test_page_call_refusals(lib):
    d = _cache()
    r = ctypes.byref(d)
    bad = gs.GS_ERR_INVALID_ARG
    assert lib.gs_pages_extend(None, 0x60000, None, 1, None) == bad
    assert lib.gs_pages_extend(r, None, None, 1, None) == bad
    assert lib.gs_pages_extend(r, 0x60000, None, -1, None) == bad
    assert lib.gs_pages_extend(r, 0x60000, None, 8193, None) == gs.GS_ERR_UNSUPPORTED
    assert lib.gs_pages_fork(r, 0x60000, None, 1, None) == bad
    assert lib.gs_pages_compact(r, None, 0x60000, None, None) == bad
    assert lib.gs_kv_write(r, 2, 0x60000, 0x60000, 128, 64, 1, 0x60000, 0x60000, 1, None) == bad
    assert lib.gs_kv_write(r, 0, 0x60001, 0x60000, 128, 64, 1, 0x60000, 0x60000, 1, None) == bad
    assert lib.gs_kv_write(r, 0, 0x60000, 0x60000, -1, 64, 1, 0x60000, 0x60000, 1, None) == bad
    for call in (lambda: lib.gs_pages_extend(r, None, None, 0, None),     # nothing to do
                 lambda: lib.gs_pages_fork(r, None, None, 0, None),
                 lambda: lib.gs_pages_free(r, None, 0, None),
                 lambda: lib.gs_kv_write(r, 0, None, None, 0, 0, 0, None, None, 0, None)):
        assert call() == gs.GS_OK
    n = ctypes.c_int64(0)
    assert lib.gs_pages_workspace(r, ctypes.byref(n)) == gs.GS_OK and n.value > 0
    assert lib.gs_pages_workspace(r, None) == bad
    d.workspace_bytes = n.value - 1
    assert lib.gs_pages_fork(r, 0x60000, 0x60010, 1, None) == bad
    assert lib.gs_pages_compact(r, 0x60000, 0x60000, None, None) == bad


def _attention(d):
    a = decode.PagedAttentionArgs()
    a.cache = ctypes.pointer(d)
    a.batch, a.q_heads, a.q, a.out = 4, 8, 0x100000, 0x200000
    a.q_batch_stride = a.out_batch_stride = 512
    a.q_head_stride = a.out_head_stride = 64
    a.scale = 0.125
    a.workspace, a.workspace_bytes = 0x1000000, 1 << 30
    return a


@pytest.mark.parametrize("field,value,status", [
    ("layer", 2, gs.GS_ERR_INVALID_ARG), ("layer", -1, gs.GS_ERR_INVALID_ARG),
    ("batch", -1, gs.GS_ERR_INVALID_ARG), ("batch", 5, gs.GS_ERR_INVALID_ARG),
    ("batch", 8193, gs.GS_ERR_UNSUPPORTED), ("q_heads", 0, gs.GS_ERR_INVALID_ARG),
    ("q_heads", 3, gs.GS_ERR_INVALID_ARG), ("q", None, gs.GS_ERR_INVALID_ARG),
    ("q", 0x100001, gs.GS_ERR_INVALID_ARG), ("out", None, gs.GS_ERR_INVALID_ARG),
    ("k_new", 0x300000, gs.GS_ERR_INVALID_ARG), ("scale", float("nan"), gs.GS_ERR_INVALID_ARG),
    ("scale", float("inf"), gs.GS_ERR_INVALID_ARG), ("window", -1, gs.GS_ERR_INVALID_ARG),
    ("sinks", 4, gs.GS_ERR_INVALID_ARG), ("out_head_stride", 32, gs.GS_ERR_INVALID_ARG),
    ("q_batch_stride", -1, gs.GS_ERR_INVALID_ARG), ("workspace", None, gs.GS_ERR_INVALID_ARG),
    ("workspace_bytes", 16, gs.GS_ERR_INVALID_ARG), ("workspace", 0x1000008, gs.GS_ERR_INVALID_ARG),
])
def test_attention_refusals(lib, field, value, status):
    a = _attention(_cache())
    setattr(a, field, value)
    assert lib.gs_paged_attention(ctypes.byref(a), None) == status


def test_attention_of_no_rows_does_nothing(lib):
    a = _attention(_cache())
    a.batch = 0
    assert lib.gs_paged_attention(ctypes.byref(a), None) == gs.GS_OK
    assert lib.gs_paged_attention(None, None) == gs.GS_ERR_INVALID_ARG


def _logits():
    a = decode.GuidedLogitsArgs()
    a.batch, a.vocab, a.dtype, a.cond, a.row_stride, a.cfg = 4, 100, gs.GS_DTYPE_F32, 0x10000, 100, 1.0
    a.out, a.out_stride = 0x20000, 100
    a.workspace, a.workspace_bytes = 0x30000, 1 << 20
    return a


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, gs.GS_ERR_INVALID_ARG), ("batch", 8193, gs.GS_ERR_UNSUPPORTED),
    ("vocab", 0, gs.GS_ERR_INVALID_ARG), ("dtype", 3, gs.GS_ERR_INVALID_ARG),
    ("cond", None, gs.GS_ERR_INVALID_ARG), ("cond", 0x10002, gs.GS_ERR_INVALID_ARG),
    ("row_stride", 99, gs.GS_ERR_INVALID_ARG), ("out_stride", 99, gs.GS_ERR_INVALID_ARG),
    ("out", None, gs.GS_ERR_INVALID_ARG), ("tokens", 0x40000, gs.GS_ERR_INVALID_ARG),
    ("bias_stride", -1, gs.GS_ERR_INVALID_ARG), ("noise", 0x40002, gs.GS_ERR_INVALID_ARG),
    ("scale_lut", 0x40000, gs.GS_ERR_INVALID_ARG), ("workspace", None, gs.GS_ERR_INVALID_ARG),
    ("workspace_bytes", 8, gs.GS_ERR_INVALID_ARG),
])
def test_logits_refusals(lib, field, value, status):
    a = _logits()
    setattr(a, field, value)
    assert lib.gs_guided_logits(ctypes.byref(a), None) == status


def test_logits_step_outside_the_table_is_refused(lib):
    a = _logits()
    a.scale_lut, a.n_lut, a.step = 0x40000, 5, 5
    assert lib.gs_guided_logits(ctypes.byref(a), None) == gs.GS_ERR_INVALID_ARG
    a = _logits()
    a.batch = 0
    assert lib.gs_guided_logits(ctypes.byref(a), None) == gs.GS_OK
