"""Sizes whose indexes would pass the 32 bits that the kernels count in are refused (CPU: the
workspace queries look at sizes alone, and every call begins with the same checks)."""

import ctypes

import pytest

from bucketized_guidance_step_gb300 import build, decode, gs
from tests.test_decode_abi import _logits


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
