"""Sizes whose indexes would pass the 32 bits that the kernels count in are refused (CPU: the
workspace queries look at sizes alone, and every call begins with the same checks)."""

import ctypes

import pytest

from bucketized_guidance_step_gb300 import build, decode, gs
from tests.test_decode_abi import _attention, _cache, _logits


@pytest.fixture(scope="module")
def lib():
    build.build()
    return decode.load()


def test_a_history_row_holds_2_to_the_30_tokens_at_most(lib):
    a, n = _logits(), ctypes.c_int64(0)
    a.tokens, a.tokens_len, a.tokens_stride = 0x40000, 0x50000, 1 << 30
    assert lib.gs_guided_logits_workspace(ctypes.byref(a), ctypes.byref(n)) == gs.GS_OK
    a.tokens_stride += 1
    assert lib.gs_guided_logits_workspace(ctypes.byref(a), ctypes.byref(n)) == gs.GS_ERR_UNSUPPORTED
    assert lib.gs_guided_logits(ctypes.byref(a), None) == gs.GS_ERR_UNSUPPORTED


@pytest.mark.parametrize("layers,heads,ok", [(1 << 14, 1 << 16, True), ((1 << 14) + 1, 1 << 16, False),
                                             ((1 << 30) + 1, 1, False)])
def test_a_page_holds_2_to_the_30_layers_of_heads_at_most(lib, layers, heads, ok):
    d, n = _cache(), ctypes.c_int64(0)
    d.layers, d.kv_heads, d.page, d.dim = layers, heads, 1, 8
    want = gs.GS_OK if ok else gs.GS_ERR_UNSUPPORTED
    assert lib.gs_pages_workspace(ctypes.byref(d), ctypes.byref(n)) == want
    if not ok:
        assert lib.gs_pages_fork(ctypes.byref(d), 0x60000, 0x60010, 1, None) == want
        assert lib.gs_pages_compact(ctypes.byref(d), 0x60000, 0x60000, None, None) == want
        a = _attention(d)
        a.q_heads = heads
        assert lib.gs_paged_attention(ctypes.byref(a), None) == want
