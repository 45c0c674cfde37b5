"""Chunk attention with as many tiles as a call may have (GPU): entries without padding rows, many heads.

Tolerances are test_chunk_attention's.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from tests.chunk_reference import pool, rows_of
from tests.test_chunk_mixed import near
from tests.test_decode_attention import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dim", [(F32, 4), (BF16, 8)])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("n,new,heads", [(8192, 1, 32), (4096, 1, 64), (256, 1, 1024), (256, 1, 1023), (1024, 64, 32), (8192, 1, 31)])
def test_every_thread_counts_many_tiles(dtype, dim, n, new, heads, pad):
    k, v, table, lens, refs = pool([70, 9 + new, 130], heads=heads, dim=dim, page=16, dtype=dtype, seed=n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = decode.PagedCache(k, v, table, lens, refs, status=status)
    seq = (torch.arange(n, device="cuda") % 3).int()
    start = (torch.arange(n + 1, device="cuda") * new).int()
    g = torch.Generator(device="cuda").manual_seed(3)
    # (the queries of three entries, again and again)
    three = torch.randn((3 * new, heads, dim), generator=g, device="cuda").to(dtype)
    q = three.repeat(-(-n // 3) + 1, 1, 1)[:n * new + pad].contiguous()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    cache.chunk_attention(q, 0, seq, start, out=out, lse=lse)
    assert int(status) == 0
    for s in range(3):
        rows = rows_of(cache, q, s, s * new, new)
        near(out[s * new:(s + 1) * new], lse[s * new:(s + 1) * new], rows, dtype, dim, 6.0)
    # entries are computed in different cuts of the call: the same but for the order of sums
    used = out[:n * new].unflatten(0, (n, new)).float()
    for s in range(3):
        assert (used[s::3] - used[s]).abs().max() <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -18) * 8
    assert torch.all(out[n * new:] == 7.0) and torch.all(lse[n * new:] == 7.0)
