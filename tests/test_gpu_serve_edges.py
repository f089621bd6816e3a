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
