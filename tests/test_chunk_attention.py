"""Attention of chunks of new tokens over a paged cache (CUDA) against the oracle in float64 (GPU).

Tolerance of an output element: with w the softmax weights, A = sum w |v| and R the largest
sum of |q k| * scale of the row,
  u |out|                     the rounding to the storage type (u = 2^-8, 2^-11, 2^-24)
  + A (8 (dim + 8) 2^-24 R    the scores' fp32 sums (2^-23 a step: the tensor cores may cut instead of
                              rounding), in numerator and denominator
       + 4 (n + 64) 2^-24     the sums over n positions and their rescalings, likewise
       + u')                  the weights in 16 bits (u' = u; 0 in fp32), the sums of them are not rounded
  + n 2^-34 max |v|           fp16 weights below the normal numbers: a step of 2^-24 where the largest
                              weight is 2^9 or more
and of the log-sum-exp 4 (dim + 8) 2^-24 R + 2 (n + 64) 2^-24 + 2^-22 |lse| + 2^-20.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from oracle import decode as O
from tests.test_decode_attention import BF16, F16, F32, UNIT, build, sequence

pytestmark = pytest.mark.gpu

LEFT = 7.25                                             # what rows of no entry hold


def starts(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()


def queries(cache, tokens, group, seed=1, sd=1.5):
    heads, dim = cache.k.shape[2], cache.k.shape[4]
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, heads * group, dim), generator=g) * sd).to(cache.k.dtype).cuda()


def run(cache, q, seq, new, layer=1, **kw):
    out = torch.full_like(q, LEFT)
    lse = torch.full(q.shape[:2], LEFT, dtype=F32, device="cuda")
    cache.chunk_attention(q, layer, torch.tensor(seq, dtype=torch.int32).cuda(), starts(new), out=out, lse=lse, **kw)
    return out, lse


def visible(pos, window, sinks):
    return [j for j in range(pos + 1) if window == 0 or j < sinks or j > pos - window]


def check(cache, layer, q, out, lse, seq, new, *, scale=None, window=0, sinks=0, rows=None):
    """rows: per entry the rows that are looked at (default all)."""
    torch.cuda.synchronize()
    dt, dim = cache.k.dtype, q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    lens = cache.lens.tolist()
    got, gl, qd = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    at = 0
    for i, (s, m) in enumerate(zip(seq, new)):
        n = lens[s]
        k, v = sequence(cache, layer, s, n)
        for x in (range(m) if rows is None else rows[i]):
            b, pos = at + x, n - m + x
            keep = visible(pos, window, sinks)
            if not keep:
                assert np.all(np.isneginf(gl[b])) and np.all(got[b] == 0), (i, x)
                continue
            want, wl, A, R = O.attention(qd[b], k[keep], v[keep], scale)
            c = len(keep)
            tol = UNIT[dt] * np.abs(want) + A * (8 * (dim + 8) * 2.0 ** -24 * R[:, None] + 4 * (c + 64) * 2.0 ** -24
                                                 + (UNIT[dt] if dt != F32 else 0.0)) + 1e-30
            if dt == F16:
                tol = tol + 2.0 ** -25 + c * 2.0 ** -34 * np.abs(v[keep]).max()
            assert np.all(np.abs(got[b] - want) <= tol), (i, x, pos, np.max(np.abs(got[b] - want) / tol))
            tl = 4 * (dim + 8) * 2.0 ** -24 * R + 2 * (c + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(wl) + 2.0 ** -20
            assert np.all(np.abs(gl[b] - wl) <= tl), (i, x, pos, np.max(np.abs(gl[b] - wl) / tl))
        at += m
    assert np.all(got[at:] == LEFT) and np.all(gl[at:] == LEFT)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim", [8, 16, 24, 64, 80, 96, 104, 128, 136, 192, 256])
def test_types_and_head_sizes(dtype, dim):
    cache = build([0, 1, 5, 16, 17, 70, 131, 300], dim=dim, dtype=dtype, seed=dim)
    seq, new = [1, 2, 5, 6, 3, 7, 4], [1, 5, 3, 131, 0, 40, 1]
    q = queries(cache, sum(new) + 3, 2)
    check(cache, 1, q, *run(cache, q, seq, new), seq, new)


@pytest.mark.parametrize("dim", [4, 12, 20, 100, 252])
def test_head_sizes_of_a_few_fp32_values(dim):
    cache = build([9, 70, 300], dim=dim, dtype=F32, heads=3, page=7, seed=dim)
    seq, new = [2, 0, 1], [9, 9, 33]
    q = queries(cache, sum(new), 5)
    check(cache, 1, q, *run(cache, q, seq, new), seq, new)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 16), (3, 5), (2, 8), (5, 3), (1, 33), (16, 1), (2, 12), (1, 300)])
def test_head_layouts(dtype, heads, group):
    cache = build([3, 64, 200], heads=heads, dim=64, dtype=dtype, seed=heads * group)
    seq, new = [2, 0, 1], [21, 3, 17]
    q = queries(cache, sum(new), group)
    check(cache, 1, q, *run(cache, q, seq, new), seq, new)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (F32, 128), (BF16, 64), (BF16, 256)])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 128, 200, 512])
def test_pages_that_end_inside_a_unit(dtype, dim, page):
    cache = build([1, 63, 64, 65, 129, 700], page=page, dtype=dtype, dim=dim, seed=page)
    seq, new = [0, 1, 2, 3, 4, 5], [1, 63, 2, 30, 129, 5]
    q = queries(cache, sum(new), 4)
    check(cache, 0, q, *run(cache, q, seq, new, layer=0), seq, new)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("new", [[1, 0, 2, 70], [300, 1, 7, 33]])
def test_long_sequences_split_and_join(dtype, new):
    cache = build([5000, 1, 2049, 3333], dtype=dtype, dim=64, page=64, seed=5)
    seq = [0, 1, 2, 3]
    q = queries(cache, sum(new), 3)
    first = run(cache, q, seq, new)
    check(cache, 1, q, *first, seq, new, rows=[sorted({0, m // 2, m - 1} & set(range(m))) for m in new])
    again = run(cache, q, seq, new)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])   # not by timing


@pytest.mark.parametrize("dtype,page", [(BF16, 16), (F16, 24), (F32, 16), (BF16, 200)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (100, 5), (128, 130), (500, 1), (5000, 4), (1 << 30, 1 << 30)])
def test_windows(dtype, page, window, sinks):
    cache = build([700, 130, 20, 1, 1500], dtype=dtype, page=page, dim=64, seed=window)
    seq, new = [0, 1, 2, 3, 4], [150, 130, 3, 1, 2]
    q = queries(cache, sum(new), 2)
    rows = [sorted({0, 1, 63, 64, m - 2, m - 1} & set(range(m))) for m in new]
    check(cache, 1, q, *run(cache, q, seq, new, window=window, sinks=sinks), seq, new, window=window, sinks=sinks, rows=rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_before_the_first_token_are_empty(dtype):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = build([5, 0, 40], dtype=dtype, seed=3, status=status)
    seq, new = [0, 1, 2], [200, 9, 40]
    q = queries(cache, sum(new), 2)
    check(cache, 1, q, *run(cache, q, seq, new), seq, new)
    assert int(status) == decode.GS_DEV_BAD_SEQ


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0, 1e-30])
def test_scales(dtype, scale):
    cache = build([90, 300], dtype=dtype, seed=8)
    seq, new = [1, 0], [20, 90]
    q = queries(cache, sum(new), 2)
    check(cache, 1, q, *run(cache, q, seq, new, scale=scale), seq, new, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_scores_that_rise_and_fall_by_hundreds(dtype):
    """The reference of the softmax moves by far, up in one row and down in another."""
    cache = build([1000], dtype=dtype, dim=64, seed=2, poison=False)
    ramp = torch.linspace(-30, 30, 1000, device="cuda")
    for t in range(1000):
        cache.k[1, cache.table[0, t // 16], :, t % 16] = ramp[t].to(dtype)
    q = queries(cache, 200, 2)
    q[::2] = q[::2].abs()
    q[1::2] = -q[1::2].abs()
    check(cache, 1, q, *run(cache, q, [0], [200]), [0], [200], rows=[[0, 1, 2, 3, 100, 101, 198, 199]])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_largest_values_stay_finite(dtype):
    cache = build([400], dtype=dtype, dim=64, seed=2, poison=False)
    cache.v.fill_(3e4)
    cache.k.fill_(0.5)
    q = queries(cache, 300, 1)
    out, lse = run(cache, q, [0], [300])
    torch.cuda.synchronize()
    assert torch.all((out[:300].double() - cache.v.flatten()[0].double()).abs() <= 3e4 * (UNIT[dtype] * 2 + 2.0 ** -20))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_what_later_tokens_hold_does_not_reach_earlier_rows(dtype, bad, which):
    cache = build([200, 500], dtype=dtype, dim=64, page=16, seed=11)
    seq, new = [0, 1], [150, 60]
    q = queries(cache, sum(new), 2)
    want = run(cache, q, seq, new)
    x = cache.k if which == "k" else cache.v
    for s, t in ((0, 120), (1, 499)):                   # rows from 70 and from 59 on see them
        x[1, cache.table[s, t // 16], 1, t % 16, 5] = bad
    got = run(cache, q, seq, new)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o[:70], w[:70]) and torch.equal(o[150:209], w[150:209])
        assert torch.equal(o[:, :2], w[:, :2])          # the other kv head's
    if which == "v":
        assert not torch.isfinite(got[0][70:150, 2:, 5].double()).any()
        assert torch.equal(got[0][70:150, 2:, 6], want[0][70:150, 2:, 6])
    # a window that has left the position behind is not reached either
    a, b = run(cache, q, seq, new, window=20), None
    x[1, cache.table[0, 120 // 16], 1, 120 % 16, 5] = 0.5
    b = run(cache, q, seq, new, window=20)
    torch.cuda.synchronize()
    for o, w in zip(a, b):
        assert torch.equal(o[90:150], w[90:150])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["gap", "heads_first", "odd", "one_query"])
def test_strides_of_queries_and_outputs(dtype, layout):
    cache = build([90, 40], dtype=dtype, dim=64, seed=4)
    seq, new = [0, 1], [33, 40]
    q0 = queries(cache, 75, 2)

    def place(x):
        T, H, D = x.shape
        if layout == "gap":
            return torch.full((T, H + 1, D + 16), LEFT, dtype=dtype, device="cuda")[:, :H, :D]
        if layout == "heads_first":
            return torch.full((H, T, D), LEFT, dtype=dtype, device="cuda").transpose(0, 1)
        if layout == "odd":
            return torch.full((T * H * (D + 1) + 1,), LEFT, dtype=dtype, device="cuda")[1:].view(T, H, D + 1)[:, :, :D]
        return torch.full((T, H, D), LEFT, dtype=dtype, device="cuda")

    if layout == "one_query":                           # every row the same one: stride 0
        q = q0[:1].expand(75, -1, -1)
    else:
        q = place(q0)
        q.copy_(q0)
    out = place(q0)
    lse = torch.full(q0.shape[:2], LEFT, device="cuda")
    cache.chunk_attention(q, 1, torch.tensor(seq, dtype=torch.int32).cuda(), starts(new), out=out, lse=lse)
    check(cache, 1, q, out, lse, seq, new)


@pytest.mark.parametrize("order", [(0, 1, 2, 3, 4), (1, 0, 3, 2, 4), (2, 3, 0, 1, 4), (3, 1, 0, 2, 4)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_cache_layouts(order, dtype):
    cache = build([90, 340], dtype=dtype, dim=128, order=order, seed=9)
    seq, new = [0, 1], [17, 40]
    q = queries(cache, 57, 2)
    check(cache, 1, q, *run(cache, q, seq, new), seq, new)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_entries(dtype):
    """More entries than a block has threads, most of them of one token or none."""
    lens = [1 + (i * 37) % 90 for i in range(60)]
    cache = build(lens, dtype=dtype, dim=64, seed=6)
    seq = [(i * 7) % 60 for i in range(1111)]
    new = [min(lens[s], (0, 1, 1, 3)[i % 4]) for i, s in enumerate(seq)]
    new[500] = lens[seq[500]]
    q = queries(cache, sum(new) + 9, 2)
    check(cache, 1, q, *run(cache, q, seq, new), seq, new)


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (F16, 192), (F32, 32)])
@pytest.mark.parametrize("n,window", [(110, 0), (260, 70), (700, 0), (1500, 0)])
def test_many_tiles(dtype, dim, n, window):
    """More tiles than blocks, from one row to hundreds, over sequences of 1 to 900 tokens: every row is there."""
    lens = [1 + (i * 211) % 900 for i in range(25)]
    cache = build(lens, dtype=dtype, dim=dim, seed=n)
    seq = [(i * 7) % 25 for i in range(n)]
    new = [min(lens[s], (1, 3, 40, 0, 130)[i * i % 5] + i % 7) for i, s in enumerate(seq)]
    q = queries(cache, sum(new) + 2, 3)
    first = run(cache, q, seq, new, window=window)
    assert not (first[1][:sum(new)] == LEFT).any()
    rows = [sorted({0, m // 2, m - 1} & set(range(m))) if i % (n // 40) == 0 or i > n - 4 else [] for i, m in enumerate(new)]
    check(cache, 1, q, *first, seq, new, window=window, rows=rows)
    # An entry's rows alone give the same but for the order of sums.
    i = max(range(n), key=lambda i: new[i])
    at, m = sum(new[:i]), new[i]
    one = run(cache, q[at:at + m], seq[i:i + 1], [m], window=window)
    assert (one[1] - first[1][at:at + m]).abs().max() < 1e-3
    again = run(cache, q, seq, new, window=window)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_most_entries(dtype):
    cache = build([40], dtype=dtype, dim=64, heads=1, seed=6)
    n = decode.GS_MAX_SEQS
    q = queries(cache, n, 1)
    q[:] = q[:1]
    out, lse = run(cache, q, [0] * n, [1] * n)
    check(cache, 1, q[:1], out[:1], lse[:1], [0], [1])
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_flags(dtype):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def flagged(cache, seq, start, tokens=30):
        status.zero_()
        q = queries(cache, tokens, 2)
        out, lse = torch.full_like(q, LEFT), torch.full(q.shape[:2], LEFT, device="cuda")
        cache.chunk_attention(q, 1, torch.tensor(seq, dtype=torch.int32).cuda(),
                              torch.tensor(start, dtype=torch.int32).cuda(), out=out, lse=lse)
        return q, out, lse, int(status)

    cache = build([30, 50, 40], dtype=dtype, seed=1, status=status)
    q, out, lse, word = flagged(cache, [0, 1], [0, 10, 30])
    assert word == 0
    check(cache, 1, q, out, lse, [0, 1], [10, 20])
    for seq in (-1, 3, 1 << 30):                        # a sequence outside the cache reads as an empty one
        q, out, lse, word = flagged(cache, [0, seq], [0, 10, 30])
        assert word == decode.GS_DEV_BAD_SEQ
        check(cache, 1, q[:10], out[:10], lse[:10], [0], [10])
        assert torch.all(out[10:] == 0) and torch.all(torch.isneginf(lse[10:]))
    for start in ([0, 10, 5], [0, 10, 31], [0, 10, -(1 << 31)], [0, 10, (1 << 31) - 1]):    # rows that are not q's
        q, out, lse, word = flagged(cache, [0, 1], start)
        assert word == decode.GS_DEV_BAD_SEQ
        check(cache, 1, q, out, lse, [0], [10])
    q, out, lse, word = flagged(cache, [0, 1, 2], [-4, 10, 20, 30])
    assert word == decode.GS_DEV_BAD_SEQ and torch.all(out[:10] == LEFT)
    # a page outside the pool reads as zeros
    for page in (-1, cache.k.shape[1], 1 << 30):
        was = int(cache.table[1, 1])
        cache.table[1, 1] = page
        q, out, lse, word = flagged(cache, [1], [0, 30])
        assert word == decode.GS_DEV_BAD_SEQ
        cache.table[1, 1] = was
        zero = build([30, 50, 40], dtype=dtype, seed=1)
        for x in (zero.k, zero.v):
            x[:, was] = 0
        check(zero, 1, q, out, lse, [1], [30])
    cache.lens[1] = 1 << 20                             # a length past the table is cut
    cols = cache.table.shape[1]
    table = torch.arange(cols, dtype=torch.int32, device="cuda") % cache.k.shape[1]
    cache.table[1] = table
    cache.k.nan_to_num_()
    cache.v.nan_to_num_()
    q, out, lse, word = flagged(cache, [1], [0, 30])
    assert word == decode.GS_DEV_BAD_SEQ
    cache.lens[1] = cols * 16
    check(cache, 1, q, out, lse, [1], [30])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranges_that_overlap_end(dtype):
    """Against the rules: the same rows in many entries, more tiles than the call's sizes allow for."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = build([2000], dtype=dtype, dim=64, heads=1, page=64, seed=1, status=status)
    q = queries(cache, 1000, 1)
    start = torch.tensor([0, 1000] * 50, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, LEFT)
    cache.chunk_attention(q, 1, torch.zeros(99, dtype=torch.int32, device="cuda"), start, out=out)
    torch.cuda.synchronize()
    assert int(status) == decode.GS_DEV_BAD_SEQ and torch.isfinite(out.double()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_replay_and_streams(dtype):
    """A captured call follows what the tensors hold, two calls on two streams do not disturb each other."""
    cache = build([3000, 90], dtype=dtype, dim=64, page=64, seed=1)
    q = queries(cache, 40, 2)
    seq = torch.tensor([0, 1], dtype=torch.int32).cuda()
    start = starts([30, 10])
    out, lse = torch.full_like(q, LEFT), torch.full(q.shape[:2], LEFT, device="cuda")
    call = cache.prepare_chunk_attention(q, 1, seq, start, out=out, lse=lse)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for new, lens in (([30, 10], [3000, 90]), ([5, 35], [100, 90]), ([0, 40], [2999, 50])):
        start.copy_(starts(new))
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(LEFT)
        lse.fill_(LEFT)
        g.replay()
        check(cache, 1, q, out, lse, [0, 1], new, rows=[sorted({0, m - 1} & set(range(m))) for m in new])
    outs = [torch.full_like(q, LEFT) for _ in range(2)]
    calls = [cache.prepare_chunk_attention(q, 1, seq, start, out=o) for o in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_large_offsets(dtype):
    """Pages and layers past 2^31 elements."""
    dim, page, heads = 128, 64, 8
    pages = (1 << 31) // (dim * page * heads) + 3
    k, v = (torch.empty((1, pages, heads, page, dim), dtype=dtype, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    for p in table[0].tolist():
        for x in (k, v):
            x[:, p].normal_(generator=torch.Generator(device="cuda").manual_seed(p))
    cache = decode.PagedCache(k, v, table, torch.tensor([150], dtype=torch.int32, device="cuda"),
                              torch.ones(pages, dtype=torch.int32, device="cuda"))
    q = queries(cache, 20, 1)
    check(cache, 0, q, *run(cache, q, [0], [20], layer=0), [0], [20])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("append", [True, False])
def test_a_chunk_is_what_single_tokens_give(dtype, append):
    """A prompt and a chunk written at once and attended to at once, against the same tokens one after the
    other with the attention of one token; the pages are shared with a fork in between."""
    heads, dim, page = 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(4)

    def empty():
        kv = torch.full((2, 1, 40, heads, page, dim), float("nan"), dtype=dtype, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        return decode.PagedCache(kv[0], kv[1], torch.full((3, 12), -1, **i32), torch.zeros(3, **i32),
                                 torch.zeros(40, **i32), status=torch.zeros(1, **i32))

    def words(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    prompt, chunk = 45, 23
    k, v = (torch.randn((prompt + 2 * chunk, heads, dim), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((prompt + 2 * chunk, 4 * heads, dim), generator=g, device="cuda").to(dtype)
    a = empty()
    a.extend(words(0), words(prompt))
    a.write(0, k[:prompt], v[:prompt], words(0), words(0, prompt))
    outs = [a.chunk_attention(q[:prompt], 0, words(0), words(0, prompt))]
    a.fork(words(0), words(2))
    a.extend(words(2, 0), words(chunk, chunk))
    a.write(0, k[prompt:], v[prompt:], words(2, 0), words(0, chunk, 2 * chunk))
    outs.append(a.chunk_attention(q[prompt:], 0, words(2, 0), words(0, chunk, 2 * chunk)))
    got = torch.cat(outs)
    b = empty()
    for t in range(prompt):
        b.extend(words(0))
        one = b.attention(q[t:t + 1], 0, seq=words(0), k_new=k[t:t + 1], v_new=v[t:t + 1])
        _near(got[t], one[0], dtype, v)
    b.fork(words(0), words(2))
    for t in range(chunk):
        rows = torch.tensor([prompt + t, prompt + chunk + t], device="cuda")
        b.extend(words(2, 0))
        if append:
            two = b.attention(q[rows], 0, seq=words(2, 0), k_new=k[rows], v_new=v[rows])
        else:
            b.write(0, k[rows], v[rows], words(2, 0), words(0, 1, 2))
            two = b.chunk_attention(q[rows], 0, words(2, 0), words(0, 1, 2))
        _near(got[rows], two, dtype, v)
    assert int(a.status) == 0 and int(b.status) == 0


def _near(x, y, dtype, v):
    """Both within u |out| and the weights' u A of the same number; fp32 sums as above."""
    tol = float(v.double().abs().max()) * (4 * UNIT[dtype] + 2.0 ** -16)
    assert (x.double() - y.double()).abs().max() <= tol
