"""Page calls on pools in states that they refuse, and with thousands of items, on
the GPU, against the oracle (exactly)."""
import numpy as np
import pytest

from oracle import serve_oracle as S
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


@pytest.mark.parametrize("pages,share", [(8000, 0.45), (20000, 0.3), (20000, 0.55), (20000, 0.6)])
def test_thousands_of_items(pages, share):
    """More items than one pass of the planning block (1024) and than blocks of the
    other kernels (2048) take: rows named again more than a pass later, copies in
    every pass, and pages that run out after the first one."""
    rng = np.random.default_rng(pages)
    n, rows, ps = 2600, 5200, 16
    p = Pool(rows, 8, pages, ps, caches=2, seed=1)
    p.o.refs[rng.random(pages) < share] = 7                        # held by nobody named below
    p.load()
    some = lambda lo, hi, m: [int(v) for v in rng.integers(lo, hi, m)]  # noqa: E731
    first = [int(v) for v in rng.permutation(n)]
    again = first + first[:700] + [-1, rows] + first[1000:1300]
    lens = some(1, 40, n)
    ends = [lens[r] if 0 <= r < n else 3 for r in again]
    p.reserve(again, [0] * len(again), ends)
    p.check()
    # forks of every first row that got its pages, and some that did not
    children = [int(v) for v in n + rng.permutation(n)]
    parents = [int(v) for v in rng.permutation(n)]
    tokens = [int(rng.integers(0, lens[r] + 1)) for r in parents]
    tokens[5], tokens[2300], children[2500], parents[2450] = -1, 9999, children[3], children[7]
    p.fork(parents, children, tokens)
    p.check()
    # each goes on where it ended: shared pages are copied, in every pass; then too few are left
    at = np.zeros(rows, int)
    at[:n] = lens
    at[children] = np.clip(tokens, 0, 40)
    named = [int(v) for v in rng.permutation(rows)[:3300]]
    named += named[:600]
    start = [int(at[r]) for r in named]
    end = [a + int(v) for a, v in zip(start, rng.integers(0, 30, len(start)))]
    p.reserve(named, start, end)
    p.check()
    held = p.o.held.copy()
    gone = some(0, rows, 2000) + some(0, rows, 2000)
    p.release(gone, some(0, 60, 4000))
    p.check()
    assert (p.o.held != held).any()
    p.compact()
    p.check()


def test_pages_run_out_in_a_later_pass():
    """Items of the first 1024 all get theirs, those of the second in part, later
    ones that need none still count as served."""
    p = Pool(rows=3000, width=4, pages=1500, caches=1)
    end = [16] * 3000
    end[2500] = 0
    assert p.o.reserve(list(range(3000)), [0] * 3000, end) == S.NO_PAGE
    assert p.o.held[:1500].all() and not p.o.held[1500:].any()
    p.o.held[:], p.o.table[:], p.o.refs[:] = 0, -1, 0
    p.reserve(None, [0] * 3000, end)
    p.check()
