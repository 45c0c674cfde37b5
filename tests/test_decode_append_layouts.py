"""Appends where runs cross pages, with windows and sinks, and in wide heads; windows over odd pages
(GPU). Tolerances are those at the head of test_decode_attention.py."""

import pytest
import torch
from tests.test_decode_attention import BF16, F16, F32, build, check, queries, run

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int32 if x.dtype == F32 else torch.int16)


def append(dtype, dim, group, page, window, sinks, lens, order):
    cache = build(lens, dtype=dtype, dim=dim, page=page, seed=page + dim, order=order)
    n = len(lens)
    q = queries(cache, n, group)
    qkv = torch.randn((n, 4 * dim + 7), generator=torch.Generator().manual_seed(9)).to(dtype).cuda()
    k_new, v_new = qkv[:, 3:3 + 2 * dim].view(n, 2, dim), qkv[:, 5 + 2 * dim:5 + 4 * dim].view(n, 2, dim)
    before = cache.k.clone(), cache.v.clone()
    out, lse = run(cache, q, k_new=k_new, v_new=v_new, window=window, sinks=sinks)
    torch.cuda.synchronize()
    for s, length in enumerate(lens):
        if length:
            p, r = int(cache.table[s, (length - 1) // page]), (length - 1) % page
            before[0][1, p, :, r], before[1][1, p, :, r] = k_new[s], v_new[s]
    for now, was in zip((cache.k, cache.v), before):                  # stored there, and nowhere else
        assert torch.equal(bits(now), bits(was))
    check(cache, 1, q, out, lse, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("page", [1, 5, 8, 16, 24])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 4), (100, 70)])
def test_append(dtype, page, window, sinks):
    append(dtype, 64, 3, page, window, sinks, [1, 16, 17, 0, 64, 65, 330], (0, 1, 3, 2, 4))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,group", [(256, 2), (256, 9), (136, 4), (96, 16), (8, 1)])
@pytest.mark.parametrize("page,window,sinks", [(24, 0, 0), (7, 50, 3)])
def test_append_in_other_heads(dtype, dim, group, page, window, sinks):
    append(dtype, dim, group, page, window, sinks, [1, 30, 0, 200], (0, 1, 2, 3, 4))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [3, 8, 24])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (64, 0), (100, 70), (5, 400)])
def test_window_and_sinks_over_odd_pages(dtype, page, window, sinks):
    cache = build([0, 1, 5, 16, 99, 171, 405], dtype=dtype, dim=64, page=page, seed=window)
    q = queries(cache, 7, 2)
    check(cache, 1, q, *run(cache, q, window=window, sinks=sinks), window=window, sinks=sinks)
