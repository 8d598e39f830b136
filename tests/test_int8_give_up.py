"""What the int8 linear layer does when a wait runs out: with a limit of 1 ns no
epilogue waits as long as its tile's products take, whatever the kernel or the
split.  Every kernel then gives up by itself (every wait is bounded; nothing is
left out and nothing faults), the status says so, nothing is written that is
not right, and the next call is right."""
import pytest
import torch

import dora_adapter_factored_b200 as dora
from dora_adapter_factored_b200 import _abi

pytestmark = pytest.mark.gpu

# Long products (k-blocks of at least a quarter of a microsecond each), one shape
# for each kernel and split, partials behind the ring and over it.
SHAPES = {
    ("tile", 1, 0): (64, 128 * 256, 4096),
    ("tile", 2, 0): (24, 8192, 8192),
    ("tile", 4, 0): (9, 2500, 12288),
    ("tile", 4, 1): (5, 4824, 16384),
    ("tile", 8, 0): (64, 128, 32768),
    ("tile", 8, 1): (3, 2316, 32768),
    ("pair", 1, 0): (1500, 4096, 4096),
    ("pair", 2, 0): (333, 2048, 8192),
    ("pair", 2, 1): (199, 5677, 23088),
    ("pair", 4, 0): (1063, 200, 14800),
    ("pair", 4, 1): (172, 2341, 87584),
}


def _form(shape, device=(0, 0, 0)):
    p = dora.dora_linear_i8_plan(*shape, *device)
    return (("dot", "tile", "pair")[p["kernel"]], p["splits"], p["partials_over_ring"])


@pytest.mark.parametrize("form", SHAPES, ids=str)
def test_every_form_gives_up_when_a_wait_runs_out(form):
    shape = SHAPES[form]
    assert _form(shape) == form
    T, d_out, d_in = shape
    g = torch.Generator("cuda").manual_seed(T + d_out)
    codes = lambda r, c: torch.randint(-128, 128, (r, c), dtype=torch.int8, device="cuda",
                                       generator=g)
    xq, wq = codes(T, d_in), codes(d_out, d_in)
    sx, sw = torch.rand(T, device="cuda", generator=g) + 0.5, \
        torch.rand(d_out, device="cuda", generator=g) + 0.5
    ref = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
    assert dora.dora_get_device_status() == _abi.DORA_OK
    unwritten = -12345.5
    for _ in range(3):
        y = torch.full_like(ref, unwritten)
        dora.dora_set_wait_timeout_ns(1)
        try:
            dora.dora_linear_i8(xq, sx, wq, sw, y=y)
            status = dora.dora_get_device_status()
        finally:
            dora.dora_set_wait_timeout_ns(0)
        assert status == _abi.DORA_ERR_TIMEOUT
        assert bool((y == unwritten).any())
        assert bool(((y == unwritten) | (y == ref)).all())
        again = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
        assert dora.dora_get_device_status() == _abi.DORA_OK
        assert torch.equal(again, ref)


def test_a_limit_that_is_long_enough_changes_nothing():
    """Limits below 0.1 s are kept by timed tries alone."""
    xq = torch.ones(333, 8192, dtype=torch.int8, device="cuda")
    wq = torch.ones(2048, 8192, dtype=torch.int8, device="cuda")
    s, w = torch.ones(333, device="cuda"), torch.ones(2048, device="cuda")
    dora.dora_set_wait_timeout_ns(50_000_000)
    try:
        y = dora.dora_linear_i8(xq, s, wq, w, dtype=torch.float32)
        assert dora.dora_get_device_status() == _abi.DORA_OK
    finally:
        dora.dora_set_wait_timeout_ns(0)
    assert bool((y == 8192.0).all())


SPLIT = [form for form in SHAPES if form[1] > 1]


@pytest.mark.parametrize("form", SPLIT, ids=str)
def test_no_sum_of_a_split_k_is_stored_incomplete(form):
    """Limits about as long as the products: some of the CTAs that share a tile's
    k give up and others do not.  What the tile stores is right or nothing."""
    T, d_out, d_in = SHAPES[form]
    g = torch.Generator("cuda").manual_seed(d_in)
    codes = lambda r, c: torch.randint(-128, 128, (r, c), dtype=torch.int8, device="cuda",
                                       generator=g)
    xq, wq = codes(T, d_in), codes(d_out, d_in)
    sx, sw = torch.rand(T, device="cuda", generator=g) + 0.5, \
        torch.rand(d_out, device="cuda", generator=g) + 0.5
    ref = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
    assert dora.dora_get_device_status() == _abi.DORA_OK
    unwritten = -12345.5
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(ref)
    try:
        for step in range(48):
            flush.zero_()  # the operands come from memory, not from L2
            y.fill_(unwritten)
            torch.cuda.synchronize()
            dora.dora_set_wait_timeout_ns(int(500 * 1.1 ** step))  # 0.5 to 44 us
            dora.dora_linear_i8(xq, sx, wq, sw, y=y)
            status = dora.dora_get_device_status()
            right = y == ref
            assert bool((right | (y == unwritten)).all()), f"step {step}"
            assert status in (_abi.DORA_OK, _abi.DORA_ERR_TIMEOUT)
            assert status == _abi.DORA_ERR_TIMEOUT or bool(right.all())
    finally:
        dora.dora_set_wait_timeout_ns(0)
