"""Chunk attention whose weights enter the product with V as sums of two 16-bit numbers (GPU; the refusals on the CPU).

Tolerances are test_chunk_attention's with the weights' error 2^-15 (bf16: the first number is cut to 8 bits, 2^-7 of
the weight are left and rounded, 2^-8 of them) and 2^-21 (fp16: 2^-10 and 2^-11), and in fp16 twice its term for
weights below the normal numbers.
"""

import ctypes

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import build as builder
from bucketized_guidance_step_gb300 import decode, gs
from tests.chunk_reference import pool, rows_of
from tests.test_chunk_abi import _args
from tests.test_decode_abi import _cache
from tests.test_decode_attention import BF16, F16, F32, UNIT, build

WEIGHTS = {BF16: 2.0 ** -15, F16: 2.0 ** -21, F32: 0.0}
LEFT = 7.25


def check(cache, q, seq, new, *, layer=0, scale=None, window=0, sinks=0, some=None, split=True):
    """Runs the call and returns its outputs; `some`: the entries that are looked at."""
    dt, dim = q.dtype, q.shape[2]
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    out, lse = torch.full_like(q, LEFT), torch.full(q.shape[:2], LEFT, device="cuda")
    cache.chunk_attention(q, layer, torch.tensor(seq, dtype=torch.int32).cuda(), start, out=out, lse=lse, scale=scale,
                          window=window, sinks=sinks, split_weights=split)
    largest = float(torch.nan_to_num(cache.v.float()).abs().max())
    for i, (s, m) in enumerate(zip(seq, new)):
        if m == 0 or (some is not None and i not in some):
            continue
        at = int(start[i])
        want, wl, R, A, count = rows_of(cache, q, s, at, m, scale=scale, window=window, sinks=sinks, layer=layer)
        c = count.double()[:, None, None]
        tol = UNIT[dt] * want.abs() + A * (8 * (dim + 8) * 2.0 ** -24 * R[..., None] + 4 * (c + 64) * 2.0 ** -24 + WEIGHTS[dt]) + 1e-30
        if dt == F16:
            tol = tol + 2.0 ** -25 + 2 * c * 2.0 ** -34 * largest
        over = ((out[at:at + m].double() - want).abs() / tol).max()
        assert over <= 1, (i, s, m, float(over))
        tl = 4 * (dim + 8) * 2.0 ** -24 * R + 2 * (c[..., 0] + 64) * 2.0 ** -24 + 2.0 ** -22 * wl.abs() + 2.0 ** -20
        assert ((lse[at:at + m].double() - wl).abs() <= tl).all()
    n = sum(new)
    assert torch.all(out[n:] == LEFT) and torch.all(lse[n:] == LEFT)
    return out, lse


def queries(cache, tokens, group, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, cache.k.shape[2] * group, cache.k.shape[4]), generator=g) * 1.5).to(cache.k.dtype).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim", [8, 64, 80, 128, 136, 256])
def test_types_and_head_sizes(dtype, dim):
    cache = build([0, 1, 5, 16, 17, 70, 131, 300], dim=dim, dtype=dtype, seed=dim)
    seq, new = [1, 2, 5, 6, 3, 7, 4], [1, 5, 3, 131, 0, 40, 1]
    check(cache, queries(cache, sum(new) + 3, 2), seq, new, layer=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page,group,window,sinks", [(16, 4, 0, 0), (24, 5, 100, 3), (1, 7, 0, 0), (200, 16, 64, 0), (33, 33, 500, 20)])
def test_pages_heads_and_windows(dtype, page, group, window, sinks):
    cache = build([700, 130, 20, 1, 1500], page=page, dtype=dtype, seed=page)
    seq, new = [0, 1, 2, 3, 4], [150, 130, 3, 1, 2]
    check(cache, queries(cache, sum(new), group), seq, new, window=window, sinks=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dim,group", [(BF16, 128, 4), (F16, 64, 5), (BF16, 256, 3)])
def test_long_and_short_chunks(dtype, dim, group):
    """Chunks of 8 tokens between chunks of 40 to 200, over sequences that blocks share and join."""
    n, heads = 24, 4
    lens = [500 + (i * 1031) % 9000 for i in range(n)]
    new = [8 if i % 2 else 40 + (i * 67) % 161 for i in range(n)]
    k, v, table, lens, refs = pool(lens, heads=heads, dim=dim, page=16, dtype=dtype, seed=group)
    cache = decode.PagedCache(k, v, table, lens, refs)
    q = queries(cache, sum(new), group)
    first = check(cache, q, list(range(n)), new)
    again = check(cache, q, list(range(n)), new, some=())
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_only_the_outputs_rounding_is_left(dtype):
    """Against 64 bits the error is that of a rounded result, sqrt(1/3) of half a step at most and 5 % for the sums; with
    rounded weights the weights' own roundings, as large, come to it."""
    k, v, table, lens, refs = pool([2000], heads=4, dim=128, page=16, dtype=dtype)
    cache = decode.PagedCache(k, v, table, lens, refs)
    q = queries(cache, 300, 4)
    want = rows_of(cache, q, 0, 0, 300)[0]
    off = [float((check(cache, q, [0], [300], split=split, some=())[0].double() - want).norm() / want.norm()) for split in (True, False)]
    rounded = float((want.to(dtype).double() - want).norm() / want.norm())
    assert off[0] <= 1.05 * rounded < off[1], (off, rounded)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_what_a_chunk_and_single_tokens_give(dtype):
    """The same tokens one after the other with the attention of one token: both as far from the reference as their
    weights may be, and a rounding of the output each."""
    cache = build([90, 333], dtype=dtype, seed=4)
    seq, new = [0, 1], [60, 60]
    q = queries(cache, 120, 4)
    out, _ = check(cache, q, seq, new, layer=1)
    refs = [rows_of(cache, q, s, 60 * s, 60, layer=1) for s in seq]
    lens = cache.lens.clone()
    for t in range(0, 60, 7):
        cache.lens.copy_(lens - 59 + t)
        one = cache.attention(q[[t, 60 + t]], 1)
        cache.lens.copy_(lens)
        for s in seq:
            want, _, R, A, count = (x[t] for x in refs[s])
            tol = 2 * UNIT[dtype] * want.abs() + A * (16 * 72 * 2.0 ** -24 * R[:, None] + 8 * (int(count) + 64) * 2.0 ** -24 + 2 * WEIGHTS[dtype])
            if dtype == F16:
                tol = tol + 2.0 ** -24 + 4 * int(count) * 2.0 ** -34 * 6
            assert ((out[60 * s + t].double() - one[s].double()).abs() <= tol).all()


@pytest.mark.gpu
def test_fp32_is_as_it_is():
    cache = build([90, 340], dtype=F32, seed=9)
    q = queries(cache, 57, 2)
    a = check(cache, q, [0, 1], [17, 40], split=True, some=())
    b = check(cache, q, [0, 1], [17, 40], split=False, some=())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_later_tokens_hold_does_not_reach_earlier_rows(dtype, bad):
    cache = build([200, 500], dtype=dtype, dim=64, page=16, seed=11)
    seq, new = [0, 1], [150, 60]
    q = queries(cache, 210, 2)
    want = check(cache, q, seq, new, layer=1)
    for s, t in ((0, 120), (1, 499)):                   # rows from 70 and from 59 on see them
        cache.v[1, cache.table[s, t // 16], 1, t % 16, 5] = bad
    got = check(cache, q, seq, new, layer=1, some=())
    for o, w in zip(got, want):
        assert torch.equal(o[:70], w[:70]) and torch.equal(o[150:209], w[150:209]) and torch.equal(o[:, :2], w[:, :2])
    assert not torch.isfinite(got[0][70:150, 2:, 5].double()).any()
    assert torch.equal(got[0][70:150, 2:, 6], want[0][70:150, 2:, 6])


@pytest.mark.gpu
def test_replay():
    cache = build([3000, 90], dtype=BF16, page=64, seed=1)
    q = queries(cache, 40, 2)
    start = torch.tensor([0, 30, 40], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    call = cache.prepare_chunk_attention(q, 1, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), start, out=out,
                                         lse=lse, split_weights=True)
    call()
    first = out.clone(), lse.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.fill_(LEFT)
    g.replay()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("value,status", [(-1, gs.GS_ERR_INVALID_ARG), (2, gs.GS_ERR_INVALID_ARG), (1 << 30, gs.GS_ERR_INVALID_ARG)])
def test_refusals(value, status):
    builder.build()
    a = _args(_cache())
    a.split_weights = value
    assert decode.load().gs_chunk_attention(ctypes.byref(a), None) == status
