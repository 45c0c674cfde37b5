"""Chunk attention calls of more than 0.2 s, the least that a wait may last (GPU).

Tolerances are test_chunk_attention's.
"""

import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from tests.chunk_reference import pool, rows_of
from tests.test_chunk_mixed import near
from tests.test_decode_attention import BF16, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,tokens,past", [(BF16, 1 << 18, 0), (F32, 1 << 15, 1 << 14), (BF16, 40, 1 << 22)])
def test_prompts_read_at_once(dtype, tokens, past):
    """(The last is short: the longest sequence, a share of a tile a block.)"""
    heads, group, dim, page = (8, 4, 128, 64) if past < 1 << 20 else (1, 6, 128, 64)
    n = tokens + past
    k, v, table, lens, refs = pool([n], heads=heads, dim=dim, page=page, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = decode.PagedCache(k, v, table, lens, refs, status=status)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((tokens, heads * group, dim), generator=g, device="cuda").to(dtype)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    start = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    cache.chunk_attention(q, 0, torch.zeros(1, dtype=torch.int32, device="cuda"), start, out=out, lse=lse)
    assert int(status) == 0 and not (lse == 7.0).any()
    for upto in (16, tokens):                           # of the entry's rows up to these the last few
        few = min(4, upto)
        part = decode.PagedCache(k, v, table, torch.tensor([past + upto], dtype=torch.int32, device="cuda"), refs)
        rows = rows_of(part, q, 0, upto - few, few)
        near(out[upto - few:upto], lse[upto - few:upto], rows, dtype, dim, 7.0)
