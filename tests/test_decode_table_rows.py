"""What stands in whole table rows after forks and frees (GPU)."""

import pytest

from tests.test_decode_pages import Both

pytestmark = pytest.mark.gpu


def test_whole_table_rows_after_forks_and_frees():
    """Columns past a forked or freed sequence's pages are -1, not only those that are read."""
    b = Both(pages=12, page=4, seqs=8, cols=6)

    def whole():
        b.check()
        assert b.table.tolist() == b.pool.table

    b.extend([0, 1, 2], [15, 8, 1])
    whole()
    b.fork([0, 1, 2], [3, 4, 5])
    whole()
    b.fork([2, 4], [3, 0])                             # shorter ones over longer ones
    whole()
    b.free([1, 5, 1])
    whole()
    b.extend([6, 7], [24, 1])                          # the first is refused, and so the second
    whole()
    b.extend([6], [9])
    b.fork([2, 2, 2, 2, 2], [7, 1, 5, 3, 0])           # some find no page: empty
    whole()
    assert b.pool.no_page and not b.pool.bad
    b.free([0, 1, 2, 3, 4, 5, 6, 7])
    whole()
    assert not b.refs.any()
