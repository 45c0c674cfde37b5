"""States that no call makes and lists that fit nothing: flagged, and nothing else is touched (GPU)."""

import pytest
import torch

from bucketized_guidance_step_gb300 import decode
from tests.test_decode_pages import F32, Both
from tests.test_decode_refused_stores import BF16, attend, make, new_tokens, word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [5, 16])
@pytest.mark.parametrize("length", [2 ** 20, 2 ** 31 - 1])
def test_append_past_the_table_stores_nothing(page, length):
    """The row is cut to what the table can hold; its last token there is not the new one's place."""
    c = make(3, page, 1, 2)
    c.extend(c.refs.new_tensor([0]), c.refs.new_tensor([2 * page]))
    plain, before = attend(c, [0], 3), (c.k.clone(), c.v.clone())
    assert word(c) == 0
    c.lens.fill_(length)
    got = attend(c, [0], 3, *new_tokens(1, BF16))
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1]) and word(c) == decode.GS_DEV_BAD_SEQ
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("page", [5, 16])
def test_append_to_a_page_outside_the_pool_reads_zeros(page):
    """As without the append: rows of such a page read as zeros, the new token's too."""
    c = make(3, page, 1, 2)
    c.extend(c.refs.new_tensor([0]), c.refs.new_tensor([page + 2]))
    c.table[0, 1] = 7
    plain, before = attend(c, [0], 3), (c.k.clone(), c.v.clone())
    assert word(c) == decode.GS_DEV_BAD_SEQ
    got = attend(c, [0], 3, *new_tokens(1, BF16))
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1]) and word(c) == decode.GS_DEV_BAD_SEQ
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("length", [-1, -2 ** 31, 33, 2 ** 31 - 1])
def test_free_leaves_a_sequence_whose_length_is_none(length):
    b = Both(page=8, cols=4)
    b.extend([0, 1], [20, 9])
    table, refs = b.table.clone(), b.refs.clone()
    b.lens[0] = length
    b.cache.free(b.dev([0, 1, 0]))
    torch.cuda.synchronize()
    assert b.lens.tolist()[:2] == [length, 0] and int(b.status) == decode.GS_DEV_BAD_SEQ
    refs[table[1, :2].long()] = 0
    table[1, :2] = -1
    assert torch.equal(b.table, table) and torch.equal(b.refs, refs)
    b.lens[0] = 20                                     # put right, it can be freed
    b.cache.free(b.dev([0]))
    torch.cuda.synchronize()
    assert not b.refs.any() and (b.table == -1).all() and not b.lens.any()


@pytest.mark.parametrize("start", [[0, 3, 6], [-2, 3, 5], [-1, 1, 9]])
def test_write_flags_rows_that_are_not_there(start):
    """Rows below 0 or from `tokens` on: skipped and flagged, the others stored."""
    b = Both(dtype=F32, dim=16)
    b.extend([0, 1], [12, 12])
    k = torch.randn((5, 3, 16), generator=torch.Generator().manual_seed(1)).cuda()
    want = b.k.clone()
    for i in range(2):
        for t in range(max(start[i], 0), min(start[i + 1], 5)):
            pos = 12 - (start[i + 1] - t)
            want[0, int(b.table[i, pos // 8]), :, pos % 8] = k[t]
    b.cache.write(0, k, k, b.dev([0, 1]), b.dev(start))
    torch.cuda.synchronize()
    assert torch.equal(b.k, want) and int(b.status) == decode.GS_DEV_BAD_SEQ
