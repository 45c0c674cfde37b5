"""Workspaces of calls that are made once: only the counters at their beginning are zeroed, and the
rest may hold anything (GPU)."""

import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from tests.test_decode_attention import BF16, F32, build, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture
def memory(monkeypatch):
    """Unset int32 memory holds -1; how many words each call fills with zeros."""
    zeroed, empty, zeros, zero_ = [], torch.empty, torch.zeros, torch.Tensor.zero_

    def dirty(*a, **kw):
        t = empty(*a, **kw)
        return t.fill_(-1) if t.dtype == torch.int32 else t

    def count(*a, **kw):
        t = zeros(*a, **kw)
        zeroed.append(t.numel())
        return t

    def fill(t):
        zeroed.append(t.numel())
        return zero_(t)

    monkeypatch.setattr(torch, "empty", dirty)
    monkeypatch.setattr(torch, "zeros", count)
    monkeypatch.setattr(torch.Tensor, "zero_", fill)
    return zeroed


@pytest.mark.parametrize("dtype,heads,group,lens", [
    (BF16, 2, 4, [3000, 10, 700, 0]), (F32, 1, 1, [9000]), (BF16, 3, 33, [1, 500]), (F32, 2, 9, [2000, 2000, 5]),
])
def test_attention_of_one_call(memory, dtype, heads, group, lens):
    cache = build(lens, dtype=dtype, dim=64, page=16, heads=heads, seed=group)
    q = queries(cache, len(lens), group)
    for _ in range(3):
        out, lse = torch.empty_like(q), torch.full(q.shape[:2], float("nan"), device="cuda")
        memory.clear()
        cache.attention(q, 1, out=out, lse=lse)
        assert sum(memory) <= len(lens) * heads * group
        check(cache, 1, q, out, lse)


@pytest.mark.parametrize("B,V", [(1, 300000), (5, 40000), (70, 9000)])
def test_logits_of_one_call(memory, B, V):
    x = torch.randn((B, V), generator=torch.Generator().manual_seed(V)).cuda()
    for _ in range(3):
        memory.clear()
        out, token, logprob = decode.guided_logits(x)
        assert sum(memory) <= B
        assert torch.equal(out, x) and torch.equal(token.long(), x.argmax(1))
        want = x.double().log_softmax(1).amax(1)
        assert (logprob.double() - want).abs().max() < 1e-4
