"""Long and short chunks in one call over caches that L2 does not hold (GPU): items of one tile of rows and of two
follow each other in a block while their keys and values are still on their way.

Tolerances are test_chunk_attention's.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from tests.chunk_reference import pool, rows_of
from tests.test_decode_attention import BF16, F16, F32, UNIT

pytestmark = pytest.mark.gpu


def near(got, gl, ref, dtype, dim, v_max, weights=None):
    """weights: relative error of the weights in the product with V (default: rounded to the type)."""
    want, wl, R, A, count = ref
    u, c = UNIT[dtype], count.double()[:, None, None]
    w = (u if dtype != F32 else 0.0) if weights is None else weights
    tol = u * want.abs() + A * (8 * (dim + 8) * 2.0 ** -24 * R[..., None] + 4 * (c + 64) * 2.0 ** -24 + w) + 1e-30
    if dtype == F16:
        tol = tol + 2.0 ** -25 + c * 2.0 ** -34 * v_max
    over = ((got.double() - want).abs() / tol).max()
    assert over <= 1, float(over)
    tl = 4 * (dim + 8) * 2.0 ** -24 * R + 2 * (c[..., 0] + 64) * 2.0 ** -24 + 2.0 ** -22 * wl.abs() + 2.0 ** -20
    assert ((gl.double() - wl).abs() <= tl).all()


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("group", [3, 4, 5, 7])
@pytest.mark.parametrize("window", [0, 1500])
def test_long_and_short_chunks(dtype, dim, group, window):
    """Chunks of 8 tokens (one tile) between chunks of 40 to 200 (whole tiles of two and tails of one)."""
    n, heads = 48, 8
    lens = [1500 + (i * 1031) % (2900 * 128 // dim) for i in range(n)]
    new = [8 if i % 2 else 40 + (i * 67) % 161 for i in range(n)]
    k, v, table, lens, refs = pool(lens, heads=heads, dim=dim, page=16, dtype=dtype, seed=group)
    assert k.nbytes + v.nbytes > 2 * 129 * 2 ** 20
    cache = decode.PagedCache(k, v, table, lens, refs)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    seq = torch.randperm(n, generator=torch.Generator().manual_seed(1)).int().cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    q = (torch.randn((sum(new), heads * group, dim), generator=g, device="cuda") * 1.5).to(dtype)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    call = cache.prepare_chunk_attention(q, 0, seq, start, window=window, sinks=4 if window else 0, out=out, lse=lse)
    call()
    first = out.clone(), lse.clone()
    for i, s in enumerate(seq.tolist()):
        at, m = int(start[i]), new[i]
        near(out[at:at + m], lse[at:at + m], rows_of(cache, q, s, at, m, window=window, sinks=4 if window else 0),
             dtype, dim, float(torch.nan_to_num(v.float()).abs().max()))
    for _ in range(30):
        out.fill_(7.0)
        lse.fill_(7.0)
        call()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
