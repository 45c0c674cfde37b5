"""The chunk attention's C ABI (CPU): struct layout, and the refusals that come before any CUDA call."""

import ctypes
import re
import shutil
import subprocess

import pytest

from bucketized_guidance_step_gb300 import build, decode, gs
from tests.test_decode_abi import CACHE_REFUSALS, HEADER, _cache


@pytest.fixture(scope="module")
def lib():
    build.build()
    return decode.load()


def layout_of(repo_tmp, name, struct):
    """{field: offset} and the size of a struct of the header, from a C compiler."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = [f'printf("sizeof %zu\\n", sizeof({name}));']
    lines += [f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f, _ in struct._fields_]
    src = repo_tmp / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"gs_decode.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = repo_tmp / "layout"
    subprocess.run([cc, "-std=c11", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return {k: int(v) for k, v in (line.split() for line in out.splitlines())}


def test_struct_matches_the_header(lib, repo_tmp):
    got = layout_of(repo_tmp, "gs_chunk_attention_args", decode.ChunkAttentionArgs)
    assert got["sizeof"] == ctypes.sizeof(decode.ChunkAttentionArgs)
    for f, _ in decode.ChunkAttentionArgs._fields_:
        assert got[f] == getattr(decode.ChunkAttentionArgs, f).offset, f
    text = open(HEADER).read()
    assert int(re.search(r"#define GS_CHUNK_COUNTERS\s+(\d+)", text).group(1)) == decode.GS_CHUNK_COUNTERS


def _args(d):
    a = decode.ChunkAttentionArgs()
    a.cache = ctypes.pointer(d)
    a.tokens, a.n, a.seq, a.start = 20, 3, 0x60000, 0x70000
    a.q_heads, a.q, a.out = 8, 0x100000, 0x200000
    a.q_token_stride = a.out_token_stride = 512
    a.q_head_stride = a.out_head_stride = 64
    a.scale = 0.125
    a.workspace, a.workspace_bytes = 0x1000000, 1 << 40
    return a


@pytest.mark.parametrize("field,value,status", CACHE_REFUSALS)
def test_cache_refusals(lib, field, value, status):
    d = _cache()
    setattr(d, field, value)
    assert lib.gs_chunk_attention(ctypes.byref(_args(d)), None) == status


@pytest.mark.parametrize("field,value,status", [
    ("layer", 2, gs.GS_ERR_INVALID_ARG), ("layer", -1, gs.GS_ERR_INVALID_ARG),
    ("tokens", -1, gs.GS_ERR_INVALID_ARG), ("n", -1, gs.GS_ERR_INVALID_ARG),
    ("n", 8193, gs.GS_ERR_UNSUPPORTED), ("tokens", 1 << 28, gs.GS_ERR_UNSUPPORTED),
    ("q_heads", 0, gs.GS_ERR_INVALID_ARG), ("q_heads", 3, gs.GS_ERR_INVALID_ARG),
    ("q_heads", 1 << 17, gs.GS_ERR_UNSUPPORTED), ("q", None, gs.GS_ERR_INVALID_ARG),
    ("q", 0x100001, gs.GS_ERR_INVALID_ARG), ("out", None, gs.GS_ERR_INVALID_ARG),
    ("out", 0x200001, gs.GS_ERR_INVALID_ARG), ("lse", 0x300002, gs.GS_ERR_INVALID_ARG),
    ("seq", None, gs.GS_ERR_INVALID_ARG), ("seq", 0x60002, gs.GS_ERR_INVALID_ARG),
    ("start", None, gs.GS_ERR_INVALID_ARG), ("start", 0x70001, gs.GS_ERR_INVALID_ARG),
    ("scale", float("nan"), gs.GS_ERR_INVALID_ARG), ("scale", float("inf"), gs.GS_ERR_INVALID_ARG),
    ("window", -1, gs.GS_ERR_INVALID_ARG), ("sinks", -1, gs.GS_ERR_INVALID_ARG),
    ("sinks", 4, gs.GS_ERR_INVALID_ARG), ("q_token_stride", -1, gs.GS_ERR_INVALID_ARG),
    ("q_head_stride", -1, gs.GS_ERR_INVALID_ARG), ("out_head_stride", 32, gs.GS_ERR_INVALID_ARG),
    ("out_token_stride", 32, gs.GS_ERR_INVALID_ARG), ("workspace", None, gs.GS_ERR_INVALID_ARG),
    ("workspace_bytes", 16, gs.GS_ERR_INVALID_ARG), ("workspace", 0x1000008, gs.GS_ERR_INVALID_ARG),
])
def test_refusals(lib, field, value, status):
    a = _args(_cache())
    setattr(a, field, value)
    assert lib.gs_chunk_attention(ctypes.byref(a), None) == status


def test_calls_that_do_nothing(lib):
    for field in ("tokens", "n"):
        a = _args(_cache())
        setattr(a, field, 0)
        a.q = a.out = a.seq = a.start = a.workspace = None
        assert lib.gs_chunk_attention(ctypes.byref(a), None) == gs.GS_OK
    assert lib.gs_chunk_attention(None, None) == gs.GS_ERR_INVALID_ARG


def test_workspace(lib):
    a, n = _args(_cache()), ctypes.c_int64(0)
    assert lib.gs_chunk_attention_workspace(ctypes.byref(a), None) == gs.GS_ERR_INVALID_ARG
    assert lib.gs_chunk_attention_workspace(None, ctypes.byref(n)) == gs.GS_ERR_INVALID_ARG
    assert lib.gs_chunk_attention_workspace(ctypes.byref(a), ctypes.byref(n)) == gs.GS_OK
    assert n.value >= 4 * decode.GS_CHUNK_COUNTERS
    a.workspace_bytes = n.value - 1
    assert lib.gs_chunk_attention(ctypes.byref(a), None) == gs.GS_ERR_INVALID_ARG
