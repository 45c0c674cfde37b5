"""Stores into positions that a sequence was not given: none is made (GPU).

gs_pages_extend leaves a sequence that it cannot serve at its old length. An append or a write that
follows would then meet the last tokens it holds, which other sequences may share. Nothing may be
stored there, the status word says so, and attention goes over what the cache holds: bit for bit
what the same call without the new token gives.
"""

import pytest
import torch

from bucketized_guidance_step_gb300 import decode

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LAYERS, HEADS, DIM = 2, 2, 64


def dev(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def make(pages, page, seqs, cols, dtype=BF16, seed=0):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((LAYERS, pages, HEADS, page, DIM), generator=g).to(dtype).cuda() for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    return decode.PagedCache(k, v, torch.full((seqs, cols), -1, **i32), torch.zeros(seqs, **i32),
                             torch.zeros(pages, **i32), status=torch.zeros(1, **i32))


def new_tokens(n, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((n, HEADS, DIM), generator=g).to(dtype).cuda() for _ in range(2)]


def word(cache):
    """The status word, which is then zeroed."""
    w = int(cache.status)
    cache.status.zero_()
    return w


def attend(cache, seq, group, k_new=None, v_new=None, **kw):
    g = torch.Generator().manual_seed(7)
    q = torch.randn((len(seq), HEADS * group, DIM), generator=g).to(cache.k.dtype).cuda()
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
    cache.attention(q, 1, seq=dev(seq), k_new=k_new, v_new=v_new, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,group", [(BF16, 4), (F16, 20), (F32, 3)])
@pytest.mark.parametrize("page", [5, 16, 24])
@pytest.mark.parametrize("window,sinks", [(0, 0), (7, 2)])
def test_append_after_a_refused_extension(dtype, group, page, window, sinks):
    """A child that shares its parent's full pages, and no page left for its next token."""
    c = make(3, page, 3, 4, dtype)
    c.extend(dev([0, 2]), dev([2 * page, 1]))
    c.fork(dev([0]), dev([1]))                         # full pages: shared, none taken
    assert word(c) == 0 and c.refs.tolist() == [2, 2, 1]
    before = c.k.clone(), c.v.clone()
    plain = attend(c, [1], group, window=window, sinks=sinks)
    k_new, v_new = new_tokens(1, dtype)
    c.extend(dev([1]))
    assert word(c) == decode.GS_DEV_NO_PAGE and c.lens.tolist() == [2 * page, 2 * page, 1]
    got = attend(c, [1], group, k_new, v_new, window=window, sinks=sinks)
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
    assert word(c) == decode.GS_DEV_NO_PAGE and same(got, plain)
    c.extend(dev([1]), dev([0]))                       # asks for nothing: the refusal stands
    attend(c, [1], group, k_new, v_new, window=window, sinks=sinks)
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1]) and word(c) == decode.GS_DEV_NO_PAGE
    c.free(dev([2]))                                   # room again: the next extension is served
    c.extend(dev([1]))
    attend(c, [1], group, k_new, v_new, window=window, sinks=sinks)
    assert word(c) == 0 and c.lens[1] == 2 * page + 1
    before[0][1, 2, :, 0], before[1][1, 2, :, 0] = k_new[0], v_new[0]
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])


def test_append_of_a_batch_serves_the_others():
    c = make(4, 16, 3, 4)
    c.extend(dev([0, 1, 2]), dev([16, 31, 5]))         # all four pages
    k_new, v_new = new_tokens(3, BF16)
    before = c.k.clone(), c.v.clone()
    c.extend(dev([0, 1, 2]))
    assert word(c) == decode.GS_DEV_NO_PAGE and c.lens.tolist() == [16, 32, 6]
    got = attend(c, [2, 1, 0], 2, k_new, v_new)
    assert word(c) == decode.GS_DEV_NO_PAGE
    t = c.table.tolist()
    for x, new, was in ((c.k, k_new, before[0]), (c.v, v_new, before[1])):
        was[1, t[1][1], :, 15], was[1, t[2][0], :, 5] = new[1], new[0]
        assert torch.equal(x, was)
    assert same(got, attend(c, [2, 1, 0], 2))          # the cache now holds what was attended to


def test_append_after_a_table_row_was_full():
    c = make(4, 8, 1, 2)
    c.extend(dev([0]), dev([16]))
    plain, before = attend(c, [0], 2), (c.k.clone(), c.v.clone())
    c.extend(dev([0]))
    assert word(c) == decode.GS_DEV_NO_PAGE
    got = attend(c, [0], 2, *new_tokens(1, BF16))
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
    assert word(c) == decode.GS_DEV_NO_PAGE and same(got, plain)


@pytest.mark.parametrize("page", [5, 16])
def test_append_to_a_shared_page(page):
    """A fork at a page's end, and no extension at all: the last row belongs to both."""
    c = make(4, page, 2, 3)
    c.extend(dev([0]), dev([page]))
    c.fork(dev([0]), dev([1]))
    plain, before = attend(c, [1], 4), (c.k.clone(), c.v.clone())
    got = attend(c, [1], 4, *new_tokens(1, BF16))
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
    assert word(c) == decode.GS_DEV_BAD_SEQ and same(got, plain)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_write_after_a_refused_extension(dtype):
    c = make(3, 8, 4, 4, dtype)
    c.extend(dev([0, 2]), dev([8, 5]))
    c.fork(dev([0]), dev([1]))
    c.extend(dev([3]), dev([2]))                       # takes the last page
    before = c.k.clone(), c.v.clone()
    assert word(c) == 0
    c.extend(dev([2, 1]), dev([4, 1]))                 # neither fits; 2 would need one page, 1 another
    assert word(c) == decode.GS_DEV_NO_PAGE and c.lens.tolist() == [8, 8, 5, 2]
    k, v = new_tokens(7, dtype)
    c.write(0, k, v, dev([2, 1, 3]), dev([0, 4, 5, 7]))
    t = c.table.tolist()
    before[0][0, t[3][0], :, :2], before[1][0, t[3][0], :, :2] = (x[5:7].transpose(0, 1) for x in (k, v))
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
    assert word(c) == decode.GS_DEV_NO_PAGE


def test_write_to_a_shared_page():
    c = make(4, 8, 2, 3)
    c.extend(dev([0]), dev([8]))
    c.fork(dev([0]), dev([1]))
    before = c.k.clone(), c.v.clone()
    c.write(1, *new_tokens(3, BF16), dev([1]), dev([0, 3]))
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
    assert word(c) == decode.GS_DEV_BAD_SEQ


def test_a_captured_step_stores_only_what_was_served():
    """The documented step, replayed without a look at the status word between."""
    page = 8
    c = make(3, page, 3, 4)
    c.extend(dev([0, 2]), dev([2 * page - 1, 1]))
    q = torch.randn((1, HEADS * 2, DIM), generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    k_new, v_new = new_tokens(1, BF16)
    out = torch.empty_like(q)
    extend = c.prepare_extend(dev([0]))
    attention = c.prepare_attention(q, 1, seq=dev([0]), k_new=k_new, v_new=v_new, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        extend()
        attention()
    before = c.k.clone(), c.v.clone()
    t = c.table.tolist()
    for i in range(4):                                 # served once, then refused
        graph.replay()
        torch.cuda.synchronize()
        if i == 0:
            before[0][1, t[0][1], :, page - 1], before[1][1, t[0][1], :, page - 1] = k_new[0], v_new[0]
        assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
        assert word(c) == (0 if i == 0 else decode.GS_DEV_NO_PAGE) and c.lens.tolist()[0] == 2 * page
        k_new.neg_()
    c.free(dev([2]))
    graph.replay()
    torch.cuda.synchronize()
    before[0][1, 2, :, 0], before[1][1, 2, :, 0] = k_new[0], v_new[0]
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1]) and word(c) == 0


def test_caches_over_one_table_share_a_workspace():
    """K and V of each layer in tensors of their own: extended by one, stored to by both."""
    a = make(1, 8, 1, 2)
    k, v = new_tokens(1, BF16)
    for x in ("k", "v"):
        assert getattr(a, x).shape[1] == 1
    b = decode.PagedCache(torch.zeros_like(a.k), torch.zeros_like(a.v), a.table, a.lens, a.refs,
                          status=a.status, workspace=a.workspace)
    a.extend(dev([0]), dev([8]))
    a.extend(dev([0]))
    assert word(a) == decode.GS_DEV_NO_PAGE
    b.write(0, k, v, dev([0]), dev([0, 1]))
    attend(b, [0], 1, k, v)
    assert word(a) == decode.GS_DEV_NO_PAGE and not b.k.any() and not b.v.any()
    with pytest.raises(ValueError):
        decode.PagedCache(b.k, b.v, a.table, a.lens, a.refs, workspace=a.workspace[:-1])


@pytest.mark.parametrize("how", ["free", "fork"])
def test_a_refusal_ends_with_the_sequence(how):
    """Freed, or forked onto, and given the same length again by other means: it is another one."""
    c = make(3, 8, 2, 2)
    c.extend(dev([0, 1]), dev([8, 16]))
    c.extend(dev([0]), dev([9]))
    assert word(c) == decode.GS_DEV_NO_PAGE
    if how == "free":
        c.free(dev([0]))
    else:
        c.free(dev([1]))
        c.fork(dev([1]), dev([0]))
    assert not c.lens[0] and word(c) == 0
    c.table[0, 0], c.lens[0], c.refs[0] = 0, 8, 1
    k, v = new_tokens(8, BF16)
    c.write(1, k, v, dev([0]), dev([0, 8]))
    assert word(c) == 0
    assert torch.equal(c.k[1, 0], k.transpose(0, 1)) and torch.equal(c.v[1, 0], v.transpose(0, 1))
