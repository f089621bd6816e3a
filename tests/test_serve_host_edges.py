"""The oracle of the shared pages on rows whose counts lie outside the table."""
import numpy as np
import pytest

from oracle import serve_oracle as S


@pytest.mark.parametrize("held", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_rows_with_counts_outside_the_table_are_left_as_they_are(held):
    o = S.Pool(np.full((4, 3), -1, np.int32), np.zeros(4, np.int32), np.zeros(12, np.int32), 16,
               [np.arange(12)[:, None].repeat(2, 1)])
    assert o.reserve([0, 1, 2], [0, 0, 0], [48, 33, 16]) == 0
    o.held[1] = held
    before = [a.copy() for a in (o.table, o.held, o.refs)]
    assert o.release([1, 1], [0, 40]) == S.BAD_ROW
    assert o.fork([1, 1], [3, 2], [0, 16]) == S.BAD_ROW
    assert o.reserve([1], [0], [0]) == S.BAD_ROW
    for a, b in zip((o.table, o.held, o.refs), before):
        np.testing.assert_array_equal(a, b)
    # what compaction moves is followed in as many entries as the row has
    assert o.release([0], [0]) == 0 and o.compact() == (4, S.BAD_ROW)
    assert o.table[1].tolist() == ([3, 0, 1] if held > 0 else [3, 4, 5])
