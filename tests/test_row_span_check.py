"""The row kernels' vectors of ragged rows, on the CPU, by the kernels' own index
arithmetic (dora_row_span_check walks RowSpan of csrc/quant.cuh)."""
import itertools
import random

import pytest

import dora_adapter_factored_b200 as dora
from dora_adapter_factored_b200._abi import DORA_ERR_INVALID_ARG, DORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("vec", [4, 8])
def test_ragged_rows(vec):
    widths = list(range(1, 41)) + [63, 64, 65, 100, 129, 257, 1001, 1003, 4099, 8191, 8193]
    for cols, row in itertools.product(widths, range(18)):
        dora.dora_row_span_check(vec, row, cols)


@pytest.mark.parametrize("vec", [4, 8])
def test_rows_far_into_a_matrix(vec):
    """Offsets beyond 32 bits."""
    rng = random.Random(vec)
    for _ in range(400):
        dora.dora_row_span_check(vec, rng.randrange(1 << 30), rng.randrange(1, 3000))
    for row, cols in ((1 << 30, 4099), ((1 << 30) - 1, 16383), (262144, 16383), (1, 1 << 20)):
        dora.dora_row_span_check(vec, row, cols)


def test_refusals():
    for bad in ((3, 0, 8), (8, -1, 8), (8, 0, 0)):
        with pytest.raises(dora.DoraError) as e:
            dora.dora_row_span_check(*bad)
        assert e.value.status == DORA_ERR_INVALID_ARG
    with pytest.raises(dora.DoraError) as e:
        dora.dora_row_span_check(8, 0, (1 << 20) + 1)
    assert e.value.status == DORA_ERR_UNSUPPORTED
