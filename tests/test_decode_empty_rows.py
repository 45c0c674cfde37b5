"""Attention over a batch of which most sequences are over (length 0) (GPU)."""

import pytest
import torch
from tests.test_decode_attention import BF16, F32, build, check, queries, run

pytestmark = pytest.mark.gpu


def microseconds(call):
    for _ in range(3):
        call()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(10):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 100


@pytest.mark.parametrize("live", [[0], [8191], [4000], [5, 6000], [0, 8191]])
def test_empty_rows_cost_no_chain_of_loads(live):
    """One look at a row after the other (half a microsecond each) would take milliseconds here."""
    lens = [0] * 8192
    for b in live:
        lens[b] = 900 + b % 7
    cache = build(lens, dtype=BF16, dim=64, heads=2, page=16, seed=1, layers=1)
    q = queries(cache, 8192, 1)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    assert microseconds(cache.prepare_attention(q, 0, out=out, lse=lse)) < 300
    torch.cuda.synchronize()
    pick = live + [1, 8190]
    part = cache.__class__(cache.k, cache.v, cache.table[pick].contiguous(), cache.lens[pick].contiguous(), cache.refs)
    check(part, 0, q[pick], out[pick], lse[pick])
    empty = torch.ones(8192, dtype=torch.bool)
    empty[live] = False
    assert not out[empty.cuda()].any() and torch.isneginf(lse[empty.cuda()]).all()


@pytest.mark.parametrize("dtype,group", [(BF16, 5), (F32, 3)])
@pytest.mark.parametrize("every", [2, 33, 64, 70, 500])
def test_gaps_between_live_rows(dtype, group, every):
    lens = [(b * 37) % 201 if b % every == every // 2 else 0 for b in range(1500)]
    cache = build(lens, dtype=dtype, dim=32, heads=2, page=8, seed=every, layers=1)
    q = queries(cache, 1500, group)
    check(cache, 0, q, *run(cache, q, layer=0))
    order = torch.randperm(1500, generator=torch.Generator().manual_seed(every))
    check(cache, 0, q, *run(cache, q, layer=0, seq=order.int().cuda(), window=30), rows=order.tolist(), window=30)
