"""Page calls on pools in states that they refuse, on the GPU, against the oracle
(exactly)."""
import pytest

from test_gpu_serve import Pool

pytestmark = pytest.mark.gpu

COUNTS = [-1, -2 ** 31, 5, 2 ** 31 - 1]     # of a row of 4 entries


def _rows_in_use(held):
    """Five rows of four entries; row 1's count is then `held`, all of its entries
    name pages that rows hold."""
    p = Pool(rows=5, width=4, pages=30)
    p.reserve(None, [0] * 5, [64, 64, 40, 0, 0])
    p.o.held[1] = held
    p.load()
    return p


@pytest.mark.parametrize("held", COUNTS)
@pytest.mark.parametrize("keep", [None, 0, 17, 64, 500])
def test_a_row_with_a_count_outside_the_table_is_not_released(held, keep):
    p = _rows_in_use(held)
    p.release([1, 2, 1], None if keep is None else [keep] * 3)     # (named twice)
    p.check()
    p.release([1])
    p.check()


@pytest.mark.parametrize("held", COUNTS)
def test_a_row_with_a_count_outside_the_table_is_not_forked_or_reserved(held):
    p = _rows_in_use(held)
    p.fork([1, 2, 1, 0], [3, 1, 4, 4], [20, 20, 0, 33])
    p.check()
    p.reserve([1, 2, 1], [16, 40, 0], [40, 50, 0])
    p.check()


@pytest.mark.parametrize("held", COUNTS)
def test_a_row_with_a_count_outside_the_table_is_flagged_by_compaction(held):
    """Its entries within the table follow the moves all the same."""
    p = _rows_in_use(held)
    p.release([0])
    p.check()
    p.compact()
    p.check()
    p.compact()
    p.check()


@pytest.mark.parametrize("pages", [40, 9000])
@pytest.mark.parametrize("bad", [99999, -1, 2 ** 31 - 1, -2 ** 31, 20])
def test_compaction_looks_at_the_rows_where_nothing_moves(pages, bad):
    p = Pool(rows=3, width=4, pages=pages, caches=1)
    p.reserve(None, [0] * 3, [50, 0, 20])
    p.o.table[2, 1] = bad                    # outside the pool, or (20) a free page
    p.load()
    p.compact()
    p.check()
    p.o.refs[:] = 1                          # no free page, nothing above the ones in use
    p.load()
    p.compact()
    p.check()
