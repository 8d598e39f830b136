"""The row kernels' vectors of ragged rows, on the CPU: the index arithmetic of
RowSpan (csrc/quant.cuh), restated, never loads or stores outside the matrix
and covers every element of every row once."""
import itertools

import pytest


def _span(row, cols, rows, vec):
    at = row * cols
    lead = at % vec
    base = at - lead
    vecs = (lead + cols + vec - 1) // vec
    end = base + vecs * vec > rows * cols
    return base, lead, vecs, end


@pytest.mark.parametrize("vec", [4, 8])
def test_ragged_spans_stay_inside_and_cover_each_row(vec):
    for cols, rows in itertools.product(list(range(1, 21)) + [31, 33, 100, 1003], range(1, 12)):
        for row in range(rows):
            base, lead, vecs, end = _span(row, cols, rows, vec)
            own = []
            for c in range(vecs):
                lo = lead if c == 0 else 0
                hi = min(vec, lead + cols - c * vec)
                first = base + c * vec
                assert 0 <= lo < hi <= vec
                own += range(first + lo, first + hi)
                whole = not (end and c == vecs - 1)
                # a whole vector is loaded as 16 bytes, a cut one by its own elements
                assert (first + vec if whole else first + hi) <= rows * cols
                # vectors other than the first and last are stored whole
                if 0 < c < vecs - 1:
                    assert (lo, hi) == (0, vec)
            assert own == list(range(row * cols, (row + 1) * cols))
    # rows that a block walks with a stride of whole vectors of rows start alike
    for cols, row in itertools.product(range(1, 40), range(20)):
        assert {_span(row + k * vec, cols, 400, vec)[1] for k in range(9)} == {row * cols % vec}
