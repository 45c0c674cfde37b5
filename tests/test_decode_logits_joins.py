"""Guided logits: rows of many chunks, which the block that arrives last joins (GPU)."""

import pytest
import torch

from bucketized_guidance_step_gb300 import decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,V", [(1, 1 << 20), (3, 700001), (64, 131072)])
def test_joins_of_many_chunks_repeat(B, V):
    """Every block's part is seen by the block that joins them, call after call."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn((B, V), generator=g, device="cuda")
    token = torch.empty(B, dtype=torch.int32, device="cuda")
    logprob = torch.empty(B, device="cuda")
    call = decode.prepare_guided_logits(x, token=token, logprob=logprob)
    first = None
    for i in range(60):
        at = torch.randint(0, V, (B,), generator=g, device="cuda")
        was = x.gather(1, at[:, None])
        x.scatter_(1, at[:, None], 50.0)               # this call's token, in another chunk each time
        call()
        assert torch.equal(token.long(), at) and (logprob > -1e-5).all() and (logprob <= 0).all()
        x.scatter_(1, at[:, None], was)
        call()
        got = token.clone(), logprob.clone()
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
