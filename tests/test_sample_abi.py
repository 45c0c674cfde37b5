"""The sampling operator's C ABI (CPU): struct layout, and the refusals that come before any CUDA call."""

import ctypes

import pytest
import torch

from bucketized_guidance_step_gb300 import build, decode, gs
from tests.test_chunk_abi import layout_of


@pytest.fixture(scope="module")
def lib():
    build.build()
    return decode.load()


def test_struct_matches_the_header(lib, repo_tmp):
    got = layout_of(repo_tmp, "gs_sample_args", decode.SampleArgs)
    assert got["sizeof"] == ctypes.sizeof(decode.SampleArgs)
    for f, _ in decode.SampleArgs._fields_:
        assert got[f] == getattr(decode.SampleArgs, f).offset, f


def _args():
    a = decode.SampleArgs()
    a.batch, a.vocab, a.dtype, a.logits, a.row_stride = 4, 100, gs.GS_DTYPE_BF16, 0x10000, 100
    a.token, a.logprob = 0x20000, 0x30000
    return a


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, gs.GS_ERR_INVALID_ARG), ("batch", 8193, gs.GS_ERR_UNSUPPORTED),
    ("vocab", 0, gs.GS_ERR_INVALID_ARG), ("vocab", (1 << 28) + 1, gs.GS_ERR_UNSUPPORTED),
    ("vocab", (1 << 23) + 1, gs.GS_ERR_UNSUPPORTED),
    ("dtype", 3, gs.GS_ERR_INVALID_ARG), ("logits", None, gs.GS_ERR_INVALID_ARG),
    ("logits", 0x10001, gs.GS_ERR_INVALID_ARG), ("row_stride", 99, gs.GS_ERR_INVALID_ARG),
    ("noise_stride", -1, gs.GS_ERR_INVALID_ARG), ("noise", 0x40002, gs.GS_ERR_INVALID_ARG),
    ("temperature", 0x40001, gs.GS_ERR_INVALID_ARG), ("top_k", 0x40002, gs.GS_ERR_INVALID_ARG),
    ("top_p", 0x40002, gs.GS_ERR_INVALID_ARG), ("min_p", 0x40002, gs.GS_ERR_INVALID_ARG),
    ("token", 0x20002, gs.GS_ERR_INVALID_ARG), ("logprob", 0x30001, gs.GS_ERR_INVALID_ARG),
])
def test_refusals(lib, field, value, status):
    a = _args()
    setattr(a, field, value)
    assert lib.gs_sample(ctypes.byref(a), None) == status


def test_refusals_of_calls_without_outputs_and_empty_batches(lib):
    a = _args()
    a.token = a.logprob = None
    assert lib.gs_sample(ctypes.byref(a), None) == gs.GS_ERR_INVALID_ARG
    a = _args()
    a.batch, a.logits = 0, None
    assert lib.gs_sample(ctypes.byref(a), None) == gs.GS_OK
    assert lib.gs_sample(None, None) == gs.GS_ERR_INVALID_ARG


def test_the_binding_wants_cuda_tensors(lib):
    with pytest.raises(ValueError):
        decode.sample(torch.zeros(2, 10))
    with pytest.raises(ValueError):
        decode.sample(torch.zeros(10))
