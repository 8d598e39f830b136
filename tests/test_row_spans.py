"""The row kernels' vectors of ragged rows, on the CPU: the index arithmetic of
RowSpan (csrc/quant.cuh), restated, covers every element of every row once, in
whole aligned vectors and a few loose elements, and takes the weight at the
same columns."""
import itertools

import pytest


def _span(row, cols, vec):
    lead = row * cols % vec
    head = min((vec - lead) % vec, cols)
    vecs = (cols - head) // vec
    loose = cols - vecs * vec
    return lead, head, vecs, loose


@pytest.mark.parametrize("vec", [4, 8])
def test_ragged_spans_cover_each_row_once(vec):
    for cols, rows in itertools.product(list(range(1, 21)) + [31, 33, 100, 1003], range(1, 12)):
        for row in range(rows):
            at = row * cols
            lead, head, vecs, loose = _span(row, cols, vec)
            assert 0 <= loose <= 2 * (vec - 1) < 32  # one to a lane
            assert vecs <= max(1, cols // vec)  # what a launch has room for
            own = []
            for c in range(vecs):
                first = head + c * vec
                assert (at + first) % vec == 0 and first + vec <= cols
                own += range(first, first + vec)
            own += [e if e < head else vecs * vec + e for e in range(loose)]
            assert sorted(own) == list(range(cols))
    # rows that a block walks with a stride of whole vectors of rows start alike
    for cols, row in itertools.product(range(1, 40), range(20)):
        assert len({_span(row + k * vec, cols, vec) for k in range(9)}) == 1


@pytest.mark.parametrize("vec", [4, 8])
def test_ragged_weight_is_that_of_the_vectors_columns(vec):
    for cols, row in itertools.product(list(range(1, 40)) + [1003], range(vec)):
        lead, head, vecs, _ = _span(row, cols, vec)

        def whole(v):  # the weight's columns in vector v, None past them
            assert v < 0 or v * vec >= cols or v * vec + min(vec, cols - v * vec) <= cols
            return [j if 0 <= j < cols else None for j in range(v * vec, (v + 1) * vec)]

        for c in range(vecs):
            k = c + 1 if lead else c
            got = (whole(k - 1) + whole(k))[vec - lead:2 * vec - lead]
            assert got == list(range(head + c * vec, head + (c + 1) * vec))
