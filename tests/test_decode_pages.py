"""Cache pages (CUDA) against the oracle's one-by-one bookkeeping, bit for bit (GPU)."""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from oracle.decode import Pool

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class Both:
    """A cache on the device and the oracle's pool of the same contents."""

    def __init__(self, layers=2, pages=40, heads=3, page=8, dim=64, seqs=6, cols=7, dtype=BF16,
                 seed=0, order=(0, 1, 2, 3, 4)):
        g = torch.Generator().manual_seed(seed)
        shape = (layers, pages, heads, page, dim)
        k, v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        # the same logical tensors, laid out in memory in another order of their dimensions
        back = [order.index(i) for i in range(5)]
        self.k, self.v = (x.permute(order).contiguous().cuda().permute(back) for x in (k, v))
        self.table = torch.full((seqs, cols), -1, dtype=torch.int32).cuda()
        self.lens = torch.zeros(seqs, dtype=torch.int32).cuda()
        self.refs = torch.zeros(pages, dtype=torch.int32).cuda()
        self.status = torch.zeros(1, dtype=torch.int32).cuda()
        self.cache = decode.PagedCache(self.k, self.v, self.table, self.lens, self.refs, status=self.status)
        self.pool = Pool(self.table.tolist(), [0] * seqs, [0] * pages, k.double().numpy(), v.double().numpy())

    def dev(self, x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def extend(self, seq, add):
        self.cache.extend(self.dev(seq), self.dev(add))
        self.pool.extend(seq, add)

    def fork(self, src, dst):
        self.cache.fork(self.dev(src), self.dev(dst))
        self.pool.fork(src, dst)

    def free(self, seq):
        self.cache.free(self.dev(seq))
        self.pool.free(seq)

    def check(self):
        torch.cuda.synchronize()
        assert self.lens.tolist() == self.pool.lens
        assert self.refs.tolist() == self.pool.refs
        for s, row in enumerate(self.pool.table):
            n = self.pool.held(self.pool.lens[s])
            assert self.table[s, :n].tolist() == row[:n], s
        assert np.array_equal(self.k.double().cpu().numpy(), self.pool.k)
        assert np.array_equal(self.v.double().cpu().numpy(), self.pool.v)
        word = int(self.status)
        assert bool(word & decode.GS_DEV_BAD_SEQ) == self.pool.bad
        assert bool(word & decode.GS_DEV_NO_PAGE) == self.pool.no_page


def test_extend_takes_the_lowest_free_pages_in_order():
    b = Both()
    b.extend([4, 0, 2], [17, 0, 8])
    b.check()
    assert b.table[4, :3].tolist() == [0, 1, 2] and b.table[2, :1].tolist() == [3]
    b.extend([2, 4], [1, 7])                       # a page's first row; fills the last page
    b.check()
    for _ in range(20):                            # one token each, as a decode step asks
        b.cache.extend(b.dev([0, 1, 2, 3, 4, 5]))
        b.pool.extend([0, 1, 2, 3, 4, 5], [1] * 6)
    b.check()


def test_extend_refuses_what_does_not_fit():
    b = Both(pages=5)
    b.extend([0], [9])                             # 2 pages
    b.extend([1, 2, 3, 1, 9, -1, 4], [25, 8, 0, 1, 1, 1, -2])   # 4 pages asked, 3 left; then 1
    b.check()
    assert b.pool.no_page and b.pool.bad
    b.extend([5], [7 * 8 + 1])                     # more than the table's row holds
    b.check()


@pytest.mark.parametrize("dtype,dim,page,order", [
    (BF16, 64, 8, (0, 1, 2, 3, 4)), (F32, 96, 24, (0, 1, 3, 2, 4)), (F16, 8, 1, (1, 0, 2, 3, 4)),
    (F16, 256, 16, (2, 0, 1, 3, 4)), (BF16, 80, 5, (0, 1, 3, 2, 4)),
])
def test_fork_shares_and_copies(dtype, dim, page, order):
    b = Both(dtype=dtype, dim=dim, page=page, order=order, seqs=9)
    b.extend([0, 1, 2], [3 * page + page // 2, 2 * page, 1])
    b.fork([0, 0, 1, 2, 8], [3, 4, 5, 6, 7])       # 8 is empty
    b.check()
    b.fork([0, 1, 2], [5, 3, 4])                   # into sequences that hold pages
    b.check()
    b.free([0, 6, 0])                              # listed twice
    b.check()
    b.extend([3, 5, 1], [page, 1, 2])
    b.check()


def test_fork_refuses_chains_and_lacks_of_pages():
    b = Both(pages=7, page=8)
    b.extend([0, 1], [20, 12])                     # 5 pages
    b.fork([0, 3, 0, 1, 7, 0], [3, 4, 4, 4, 5, -3])   # 3 is a destination; 4 twice; ids outside
    b.check()
    assert b.pool.bad
    b.fork([0, 1, 0], [5, 2, 4])                   # pages for some of the three only
    b.check()
    assert b.pool.no_page


@pytest.mark.parametrize("seed,pages,page", [(1, 40, 8), (2, 3000, 4), (3, 9, 16), (4, 513, 2)])
def test_compact_after_a_mixed_history(seed, pages, page):
    rng = np.random.default_rng(seed)
    b = Both(pages=pages, page=page, seqs=30, cols=12, layers=1, dim=16, heads=2, seed=seed)
    for _ in range(6):
        b.extend(rng.permutation(30)[:10].tolist(), rng.integers(0, 4 * page, 10).tolist())
        p = rng.permutation(30)
        b.fork(p[:4].tolist(), p[4:8].tolist())
        b.free(p[8:14].tolist())
    b.check()
    live = torch.zeros(1, dtype=torch.int32).cuda()
    table, refs = torch.empty_like(b.table), torch.empty_like(b.refs)
    before = b.table.clone(), b.refs.clone()
    b.cache.compact(table_out=table, refs_out=refs, live=live)      # beside the old ones
    torch.cuda.synchronize()
    assert torch.equal(b.table, before[0]) and torch.equal(b.refs, before[1])
    assert int(live) == b.pool.compact()
    b.table.copy_(table)
    b.refs.copy_(refs)
    b.check()
    b.free([0, 1, 2, 3])
    b.cache.compact()                                                # in place
    b.pool.compact()
    b.check()


@pytest.mark.parametrize("dtype,offset", [(BF16, 0), (F16, 1), (F32, 3)])
def test_write_places_ragged_prompts(dtype, offset):
    b = Both(dtype=dtype, dim=32, order=(0, 1, 3, 2, 4))
    seq, add = [3, 0, 5], [13, 1, 24]
    b.extend(seq, add)
    start = [0, 13, 14, 38]
    g = torch.Generator().manual_seed(3)
    base = torch.randn((2, 38 * 3 * 2 * 32 + offset + 8), generator=g).to(dtype).cuda()
    k, v = (x[offset:offset + 38 * 192].view(38, 3, 64)[:, :, 5:37] for x in base)   # unaligned rows
    for layer in (0, 1):
        b.cache.write(layer, k, v, b.dev(seq), b.dev(start))
        b.pool.write(layer, k.double().cpu().numpy(), v.double().cpu().numpy(), seq, start)
    b.check()
    b.cache.write(0, k, v, b.dev([3, 9]), b.dev([0, 14, 15]))       # one row too many; no such id
    b.pool.write(0, k.double().cpu().numpy(), v.double().cpu().numpy(), [3, 9], [0, 14, 15])
    b.check()


def test_refusals_of_the_binding():
    b = Both()
    with pytest.raises(ValueError):
        b.cache.extend(torch.zeros(2, dtype=torch.int64).cuda())
    with pytest.raises(ValueError):
        b.cache.extend(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.cache.fork(b.dev([0, 1]), b.dev([2]))
    with pytest.raises(ValueError):
        decode.PagedCache(b.k, b.v[:, :-1], b.table, b.lens, b.refs)
    with pytest.raises(ValueError):
        decode.PagedCache(b.k, b.v, b.table, b.lens[:-1], b.refs)
    with pytest.raises(ValueError):
        decode.PagedCache(b.k[:, :1].expand(-1, 40, -1, -1, -1), b.v, b.table, b.lens, b.refs)
    with pytest.raises(decode.GSError):
        decode.PagedCache(*(x[..., :4].contiguous() for x in (b.k, b.v)), b.table, b.lens, b.refs)


def test_a_pool_of_many_pages():
    """More pages than the bookkeeping keeps in registers (8 blocks x 512 threads x 32)."""
    pages = 150000
    b = Both(pages=pages, page=1, dim=8, heads=1, layers=1, seqs=5, cols=70000)
    b.extend([0, 1], [60000, 65000])
    b.check()
    b.fork([0, 1], [2, 3])                         # all pages full: shared only
    b.free([0])
    b.extend([4], [24999])
    b.check()
    b.extend([0], [2])                             # one page is left
    b.check()
    assert b.pool.no_page
    b.free([1, 3])
    b.cache.compact()
    b.pool.compact()
    b.check()


def test_write_of_ranges_that_do_not_rise_stays_in_its_sequence():
    b = Both(dtype=F32, dim=16)
    b.extend([0, 1], [9, 3])
    k = torch.randn((12, 3, 16)).cuda()
    before = b.k.clone()
    b.cache.write(0, k, k, b.dev([0, 1]), b.dev([0, 12, 4]))
    torch.cuda.synchronize()
    changed = (b.k != before).any(dim=4).any(dim=2)[0].nonzero()[:, 0]
    assert set(changed.tolist()) <= set(b.table[0, :2].tolist()) and int(b.status) == decode.GS_DEV_BAD_SEQ


def test_compact_leaves_an_entry_that_names_a_free_page():
    b = Both(pages=8, page=4)
    b.extend([0, 1], [4, 8])                       # pages 0; 1, 2
    b.table[1, 1] = 7                              # (a state that no call makes)
    b.refs[0] = 0
    table, refs = torch.empty_like(b.table), torch.empty_like(b.refs)
    b.cache.compact(table_out=table, refs_out=refs)
    torch.cuda.synchronize()
    assert table[1, :2].tolist() == [1, 7] and int(b.status) == decode.GS_DEV_BAD_SEQ
    assert refs.tolist() == [1, 1, 0, 0, 0, 0, 0, 0]


def test_write_of_more_prompts_than_a_block_has_threads():
    rng = np.random.default_rng(8)
    b = Both(pages=6000, page=4, dim=8, heads=1, layers=1, seqs=5000, cols=3)
    seq = rng.permutation(5000)[:4999].tolist()
    add = rng.integers(0, 4, 4999).tolist()
    b.extend(seq, add)
    start = np.concatenate([[0], np.cumsum(add)]).tolist()
    k = torch.randn((start[-1], 1, 8), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    b.cache.write(0, k, -k, b.dev(seq), b.dev(start))
    b.pool.write(0, k.double().cpu().numpy(), -k.double().cpu().numpy(), seq, start)
    b.check()
