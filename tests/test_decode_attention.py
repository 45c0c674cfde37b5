"""Attention over a paged cache (CUDA) against the oracle in float64 (GPU).

Tolerance of an output element: with w the softmax weights, A = sum w |v| and R the largest
sum of |q k| * scale of the head,
  u |out|                     the rounding to the storage type (u = 2^-8, 2^-11, 2^-24)
  + A (4 (dim + 8) 2^-24 R    the scores' fp32 sums, in numerator and denominator
       + 2 (n + 64) 2^-24     the sums over n positions and their rescalings
       + e)                   the weights as two 16-bit numbers (2^-16, 2^-22; 0 in fp32)
and of the log-sum-exp 2 (dim + 8) 2^-24 R + (n + 64) 2^-24 + 2^-22 |lse| + 2^-20.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from oracle import decode as O

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
SPLIT = {BF16: 2.0 ** -16, F16: 2.0 ** -22, F32: 0.0}


def build(lens, *, heads=2, dim=64, page=16, dtype=BF16, seed=0, layers=2, order=(0, 1, 2, 3, 4),
          extra=3, poison=True, status=None):
    """A cache whose sequences hold random pages; rows past a sequence's end hold NaN."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + extra
    cols = max(held + [1]) + 1
    perm = torch.randperm(pages, generator=g).tolist()
    shape = (layers, pages, heads, page, dim)
    k, v = (torch.full(shape, float("nan") if poison else 0.0).to(dtype) for _ in range(2))
    table = torch.full((len(lens), cols), 1 << 30, dtype=torch.int32)      # never to be followed
    refs = torch.zeros(pages, dtype=torch.int32)
    for s, n in enumerate(lens):
        for j in range(held[s]):
            p = perm.pop()
            table[s, j] = p
            refs[p] = 1
            rows = min(page, n - j * page)
            k[:, p, :, :rows] = torch.randn((layers, heads, rows, dim), generator=g).to(dtype)
            v[:, p, :, :rows] = torch.randn((layers, heads, rows, dim), generator=g).to(dtype)
    back = [order.index(i) for i in range(5)]
    k, v = (x.permute(order).contiguous().cuda().permute(back) for x in (k, v))
    return decode.PagedCache(k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             refs.cuda(), status=status)


def sequence(cache, layer, s, n):
    """K and V of a sequence's first n tokens, [n, heads, dim] in float64."""
    page = cache.k.shape[3]
    at = [(int(cache.table[s, t // page]), t % page) for t in range(n)]
    pick = [torch.stack([x[layer, p, :, r] for p, r in at]) if at else x.new_zeros((0,) + tuple(x.shape[2:5:2]))
            for x in (cache.k, cache.v)]
    return [x.double().cpu().numpy() for x in pick]


def check(cache, layer, q, out, lse, *, rows=None, scale=None, window=0, sinks=0):
    torch.cuda.synchronize()
    dt, dim = cache.k.dtype, q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    lens = cache.lens.tolist()
    got, gl, qd = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for b in range(q.shape[0]):
        s = b if rows is None else rows[b]
        n = lens[s]
        k, v = sequence(cache, layer, s, n)
        keep = O.visible(n, window, sinks)
        want, wl, A, R = O.attention(qd[b], k[keep], v[keep], scale)
        m = len(keep)
        tol = UNIT[dt] * np.abs(want) + A * (4 * (dim + 8) * 2.0 ** -24 * R[:, None]
                                             + 2 * (m + 64) * 2.0 ** -24 + SPLIT[dt]) + 1e-30
        if dt == F16:
            tol = tol + 2.0 ** -25                                   # subnormal outputs
        assert np.all(np.abs(got[b] - want) <= tol), (b, n, np.max(np.abs(got[b] - want) / tol))
        if m == 0:
            assert np.all(np.isneginf(gl[b])) and np.all(got[b] == 0)
        else:
            tl = 2 * (dim + 8) * 2.0 ** -24 * R + (m + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(wl) + 2.0 ** -20
            assert np.all(np.abs(gl[b] - wl) <= tl), (b, n)


def queries(cache, batch, group, seed=1, sd=1.5):
    heads, dim = cache.k.shape[2], cache.k.shape[4]
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((batch, heads * group, dim), generator=g) * sd).to(cache.k.dtype).cuda()


def run(cache, q, layer=1, **kw):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), dtype=F32, device="cuda")
    cache.attention(q, layer, out=out, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim", [8, 16, 24, 64, 80, 96, 104, 128, 136, 192, 256])
def test_types_and_head_sizes(dtype, dim):
    cache = build([0, 1, 5, 16, 17, 70, 131], dim=dim, dtype=dtype, seed=dim)
    q = queries(cache, 7, 2)
    check(cache, 1, q, *run(cache, q))


@pytest.mark.parametrize("dim", [4, 12, 20, 100, 252])
def test_head_sizes_of_a_few_fp32_values(dim):
    cache = build([0, 1, 9, 70, 300], dim=dim, dtype=F32, heads=3, page=7, seed=dim)
    q = queries(cache, 5, 5)
    check(cache, 1, q, *run(cache, q))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 16), (3, 5), (2, 8), (5, 3), (1, 33), (16, 1), (2, 12)])
def test_head_layouts(dtype, heads, group):
    cache = build([3, 64, 200], heads=heads, dim=64, dtype=dtype, seed=heads * group)
    q = queries(cache, 3, group)
    check(cache, 1, q, *run(cache, q))


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 512])
def test_pages_that_end_inside_a_tile(dtype, page):
    cache = build([1, 63, 64, 65, 129, 300], page=page, dtype=dtype, dim=128, seed=page)
    q = queries(cache, 6, 4)
    check(cache, 0, q, *run(cache, q, layer=0))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_long_and_short_rows_split_and_join(dtype):
    """Rows of one call from empty to thousands of positions: parts of several blocks join."""
    cache = build([0, 5000, 1, 0, 2049, 77, 3333], dtype=dtype, dim=64, page=64, seed=5)
    q = queries(cache, 7, 3)
    first = run(cache, q)
    check(cache, 1, q, *first)
    again = run(cache, q)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])   # not by timing


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (64, 0), (100, 70), (1000, 3), (5, 400)])
def test_window_and_sinks(dtype, window, sinks):
    cache = build([0, 1, 5, 16, 99, 171, 405], dtype=dtype, dim=64, page=16, seed=window)
    q = queries(cache, 7, 2)
    check(cache, 1, q, *run(cache, q, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (20, 80)])
def test_append_stores_the_new_token(dtype, group, dim):
    cache = build([1, 16, 17, 64, 1000], dtype=dtype, dim=dim, seed=group, order=(0, 1, 3, 2, 4))
    q = queries(cache, 5, group)
    g = torch.Generator().manual_seed(9)
    # rows of one projection's output: strided, and off the 16-byte boundary
    qkv = torch.randn((5, 2 * 2 * dim + 7), generator=g).to(dtype).cuda()
    k_new, v_new = qkv[:, 3:3 + 2 * dim].view(5, 2, dim), qkv[:, 5 + 2 * dim:5 + 4 * dim].view(5, 2, dim)
    before = cache.k.clone(), cache.v.clone()
    out, lse = run(cache, q, k_new=k_new, v_new=v_new)
    torch.cuda.synchronize()
    page = cache.k.shape[3]
    for s, n in enumerate(cache.lens.tolist()):
        p, r = int(cache.table[s, (n - 1) // page]), (n - 1) % page
        assert torch.equal(cache.k[1, p, :, r], k_new[s]) and torch.equal(cache.v[1, p, :, r], v_new[s])
        before[0][1, p, :, r], before[1][1, p, :, r] = k_new[s], v_new[s]
    for now, was in ((cache.k, before[0]), (cache.v, before[1])):      # nothing else is written
        assert torch.equal(now.view(torch.int16 if dtype != F32 else torch.int32),
                           was.view(torch.int16 if dtype != F32 else torch.int32))
    check(cache, 1, q, out, lse)


def test_rows_choose_their_sequences_and_strides():
    cache = build([40, 0, 7, 130], dtype=BF16, dim=64)
    rows = [3, 0, 0, 2, 1, 3]
    g = torch.Generator().manual_seed(2)
    wide = torch.randn((4, 6, 100), generator=g).to(BF16).cuda()
    q = wide.transpose(0, 1)[:, :, 9:73]                               # strided, off the boundary
    out = torch.empty((6, 70, 4), dtype=BF16, device="cuda").transpose(1, 2)[:, :, 3:67]
    assert out.stride(2) != 1
    with pytest.raises(ValueError):
        cache.attention(q, 0, out=out)
    out = torch.full((4, 6, 72), 7.0, dtype=BF16, device="cuda").transpose(0, 1)[:, :, 1:65]
    lse = torch.empty((6, 4), device="cuda")
    cache.attention(q, 0, seq=torch.tensor(rows, dtype=torch.int32).cuda(), out=out, lse=lse, scale=-0.3)
    check(cache, 0, q, out, lse, rows=rows, scale=-0.3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_values(dtype):
    """Scores far apart: the running maximum carries the sum; equal huge scores; -inf scores."""
    cache = build([200, 200, 200], dtype=dtype, dim=64, heads=1, poison=False)
    page = cache.k.shape[3]
    q = torch.zeros((3, 1, 64), dtype=dtype).cuda()
    q[:, :, 0] = 1.0
    cache.k[..., 0] = 0.0
    for t in range(200):
        cache.k[1, int(cache.table[0, t // page]), 0, t % page, 0] = 40.0 * t     # rising
        cache.k[1, int(cache.table[1, t // page]), 0, t % page, 0] = 2.0 ** 100   # all the same
        cache.k[1, int(cache.table[2, t // page]), 0, t % page, 0] = float("-inf") if t != 150 else 1.0
    out, lse = run(cache, q, scale=1.0)
    torch.cuda.synchronize()
    k, v = sequence(cache, 1, 0, 200)
    tol = 4 * UNIT[dtype] * 8
    assert np.allclose(out[0, 0].double().cpu().numpy(), v[199, 0], atol=tol, rtol=0)
    k, v = sequence(cache, 1, 1, 200)
    assert np.allclose(out[1, 0].double().cpu().numpy(), v[:, 0].mean(0), atol=tol, rtol=0)
    k, v = sequence(cache, 1, 2, 200)
    assert np.allclose(out[2, 0].double().cpu().numpy(), v[150, 0], atol=tol, rtol=0)
    assert torch.isfinite(lse).all()


def test_nan_in_a_visible_row_stays_in_its_head():
    cache = build([90, 90], dtype=BF16, dim=64, heads=2, poison=False)
    q = queries(cache, 2, 2)
    clean = run(cache, q)
    cache.k[1, int(cache.table[0, 2]), 1, 3, 5] = float("nan")
    out, lse = run(cache, q)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.equal(out[0, :2], clean[0][0, :2]) and torch.equal(out[1], clean[0][1])


def test_device_found_errors_are_flagged():
    status = torch.zeros(1, dtype=torch.int32).cuda()
    cache = build([40, 40], dtype=BF16, dim=64, status=status, poison=False)
    q = queries(cache, 2, 1)
    good = run(cache, q)
    assert int(status) == 0
    out, lse = run(cache, q, seq=torch.tensor([5, 1], dtype=torch.int32).cuda())
    assert int(status) == decode.GS_DEV_BAD_SEQ
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.equal(out[1], good[0][1])
    status.zero_()
    cache.table[0, 1] = -1                                             # a page that is none
    out, lse = run(cache, q)
    assert int(status) == decode.GS_DEV_BAD_SEQ and torch.equal(out[1], good[0][1])
    status.zero_()
    cache.lens[0] = 1 << 20                                            # past the table: cut
    run(cache, q)
    assert int(status) == decode.GS_DEV_BAD_SEQ


def test_graph_replay_and_another_stream():
    cache = build([33, 700, 1], dtype=F16, dim=128, page=16, poison=False)
    q = queries(cache, 3, 4)
    want = run(cache, q)
    out, lse = torch.empty_like(q), torch.empty((3, 8), device="cuda")
    call = cache.prepare_attention(q, 1, out=out, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        call()
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_offsets_past_32_bits():
    """A page whose first element lies past 2^31 elements into the pool."""
    pages, page, dim = (1 << 31) // (64 * 128) + 2, 64, 128
    k = torch.zeros((1, pages, 1, page, dim), dtype=BF16, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(4)
    for p in (0, pages - 1, pages - 2):
        k[0, p] = torch.randn((1, page, dim), generator=g).to(BF16).cuda()
    refs = torch.zeros(pages, dtype=torch.int32).cuda()
    refs[table[0].long()] = 1
    cache = decode.PagedCache(k, k, table, torch.tensor([150], dtype=torch.int32).cuda(), refs)
    q = queries(cache, 1, 4)
    check(cache, 0, q, *run(cache, q, layer=0))


@pytest.mark.parametrize("dtype,window", [(BF16, 0), (F32, 0), (F16, 40)])
def test_many_rows(dtype, window):
    """More rows than a warp's first look at the lengths takes, a third of them empty."""
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(-60, 130, (1100,), generator=g).clamp(min=0).tolist()
    cache = build(lens, dtype=dtype, dim=32, heads=1, page=8, seed=12, layers=1)
    q = queries(cache, 1100, 3)
    check(cache, 0, q, *run(cache, q, layer=0, window=window), window=window)
    order = torch.randperm(1100, generator=g)
    check(cache, 0, q, *run(cache, q, layer=0, window=window, seq=order.int().cuda()), rows=order.tolist(), window=window)


def test_calls_on_one_workspace_leave_it_ready():
    """The same prepared call again and again, lengths changing between: counts of arrived parts
    start from zero each time."""
    cache = build([3000, 10, 700, 0], dtype=BF16, dim=64, page=32, seed=3)
    q = queries(cache, 4, 8)
    out, lse = torch.empty_like(q), torch.empty((4, 16), device="cuda")
    call = cache.prepare_attention(q, 1, out=out, lse=lse)
    for lens in ([3000, 10, 700, 0], [1, 0, 0, 0], [2999, 1, 64, 0], [65, 9, 640, 0], [3000, 10, 700, 0]):
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for _ in range(3):
            call()
        check(cache, 1, q, out, lse)
