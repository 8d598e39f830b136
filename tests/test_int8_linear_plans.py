"""Every form of the int8 linear layer against the exact sums: which kernel,
split and ring a shape takes is asked of the library's own plan
(dora_linear_i8_plan), so that a change of the plan cannot take a form out of
the tests unseen.  On the CPU: the list below reaches all of them, on devices
with more and fewer resident clusters.  On the GPU: every output of every
shape, in both types, with and without a bias.

Tolerances as in test_parity_int8.py (u = 2^-24): without a bias the stated
fp32 operations bit for bit; with one, 2u of the product term and the last
rounding, u or half a bf16 step, 2^-8."""
import pytest
import torch

import dora_adapter_factored_b200 as dora
from dora_adapter_factored_b200 import _abi

U = 2.0 ** -24

# (T, d_out, d_in)
SHAPES = [
    # dot products: one, two, four and eight tokens, whole 16-byte rows and not
    (1, 33, 64), (2, 100, 1040), (4, 513, 272), (8, 257, 512), (3, 100, 15), (7, 129, 1003),
    # single CTAs: k whole and split, partials behind and over the ring, two an SM
    (10, 33, 64), (198, 5083, 64), (42, 33, 688), (9, 37, 400), (5, 4824, 3856),
    (18, 35, 976), (3, 2316, 12864), (700, 129, 2064),
    # ... from padded copies
    (10, 35, 65), (130, 6299, 84), (35, 34, 742), (11, 35, 392), (2, 4772, 3662), (18, 38, 908),
    (1, 2379, 14886),
    # pairs, k whole: one tile each, several, many turns of the ring, odd widths
    (1070, 33, 64), (1500, 4096, 4096), (2051, 4100, 2064), (5696, 3287, 144), (2900, 8200, 272),
    # ... token tiles in groups, the last of them narrower
    (4628, 2117, 8016), (4954, 135, 7536),
    # ... from padded copies
    (1114, 36, 73), (3000, 4113, 1025), (3921, 4789, 132), (2100, 777, 4100), (300, 9001, 1003),
    # pairs, k split two and four ways: partials behind the ring ...
    (333, 2048, 4096), (333, 4096, 14336), (1044, 35, 1760), (700, 1024, 4096), (700, 512, 8192),
    (333, 1024, 14336), (1040, 133, 6208), (1063, 200, 14800), (2825, 135, 11648),
    (1143, 130, 1761), (1063, 131, 6113),
    # ... and over it
    (199, 5677, 23088), (172, 2341, 87584), (1063, 302, 14800),
]

# (SMs, resident clusters of 4 CTAs, of 8): a B200 had 33 and 15
DEVICES = [(148, 33, 15), (148, 24, 10), (148, 28, 12), (148, 36, 18), (148, 33, 19)]

REQUIRED = {("dot",), ("pair", "persistent"), ("pair", "groups"), ("pair", "last group narrower")} \
    | {("tile", s) for s in (1, 2, 4, 8)} | {("tile", "padded"), ("tile", "two an SM")} \
    | {("tile", s, "over the ring") for s in (4, 8)} \
    | {("pair", s) for s in (1, 2, 4)} | {("pair", s, "padded") for s in (1, 2, 4)} \
    | {("pair", s, "over the ring") for s in (2, 4)}


def _forms(shape, device=(0, 0, 0)):
    """What a shape exercises."""
    p = dora.dora_linear_i8_plan(*shape, *device)
    sms = device[0] or torch.cuda.get_device_properties(0).multi_processor_count
    if p["kernel"] == 0:
        return {("dot",)}
    name = "tile" if p["kernel"] == 1 else "pair"
    tiles = p["token_tiles"] * p["channel_tiles"]
    out = {(name, p["splits"])}
    if p["padded"]:
        out |= {(name, "padded"), (name, p["splits"], "padded")}
    if p["partials_over_ring"]:
        out.add((name, p["splits"], "over the ring"))
    if name == "tile" and tiles * p["splits"] > sms:
        out.add((name, "two an SM"))
    if name == "pair":
        per_pair = tiles // (sms // 2)
        if p["splits"] == 1 and per_pair >= 4 and per_pair * p["kblocks"] > 2 * p["stages"] \
                and p["kblocks"] > 1:
            out.add((name, "persistent"))  # both accumulators again, several ring turns
        if p["group"] < p["token_tiles"]:
            out.add((name, "groups"))
            if p["token_tiles"] % p["group"]:
                out.add((name, "last group narrower"))
    return out


@pytest.mark.parametrize("device", DEVICES)
def test_the_shapes_reach_every_form(device):
    reached = set().union(*(_forms(s, device) for s in SHAPES))
    assert REQUIRED <= reached, sorted(map(str, REQUIRED - reached))


def test_plans_are_within_the_kernels_limits():
    g = torch.Generator().manual_seed(1)
    u = torch.rand(4000, 3, generator=g, dtype=torch.float64)
    for a, b, c in u.tolist():
        shape = (int(2 ** (16 * a)), int(2 ** (15 * b)), int(2 ** (4 + 13 * c)) - 1)
        for device in DEVICES[:3]:
            p = dora.dora_linear_i8_plan(*shape, *device)
            T, d_out, d_in = shape
            assert p["kernel"] in (0, 1, 2)
            if p["kernel"] == 0:
                continue
            pair = p["kernel"] == 2
            n, splits = p["tokens"], p["splits"]
            assert n % (32 if pair else 16) == 0 and 16 <= n <= (256 if pair else 128)
            assert splits in ((1, 2, 4) if pair else (1, 2, 4, 8)) and n // splits % 4 == 0
            assert p["kblocks"] == -(-d_in // 128) and splits <= p["kblocks"]
            assert n * p["token_tiles"] >= T and n * (p["token_tiles"] - 1) < T
            assert p["channel_tiles"] == -(-d_out // (256 if pair else 128))
            assert 1 <= p["stages"] <= 12
            # stages and partials fit the shared memory of a CTA
            stage = 16384 + (n // 2 if pair else n) * 128
            part = (splits - 1) * (n // splits) * 128 * 4
            room = 227 * 1024 - 1024
            assert p["stages"] * stage + (0 if p["partials_over_ring"] else part) <= room
            assert part <= room
            if pair:
                assert 1 <= p["group"] <= p["token_tiles"]


def test_plan_refusals():
    for bad in ((0, 8, 16), (1, 0, 16), (1, 8, 0)):
        with pytest.raises(dora.DoraError) as e:
            dora.dora_linear_i8_plan(*bad, *DEVICES[0])
        assert e.value.status == _abi.DORA_ERR_INVALID_ARG
    with pytest.raises(dora.DoraError):
        dora.dora_linear_i8_plan(8, 8, 16, 148, 0, 15)
    for large in (((1 << 23) + 1, 8, 16), (1, 8, dora.DORA_MAX_I8_K + 1)):
        with pytest.raises(dora.DoraError) as e:
            dora.dora_linear_i8_plan(*large, *DEVICES[0])
        assert e.value.status == _abi.DORA_ERR_UNSUPPORTED


# ------------------------------------------------------------------ GPU

@pytest.mark.gpu
def test_the_shapes_reach_every_form_on_this_device():
    reached = set().union(*(_forms(s) for s in SHAPES))
    assert REQUIRED <= reached, sorted(map(str, REQUIRED - reached))


def _operands(T, d_out, d_in):
    g = torch.Generator("cuda").manual_seed(T + 3 * d_out + 7 * d_in)
    codes = lambda r, c: torch.randint(-128, 128, (r, c), dtype=torch.int8, device="cuda",
                                       generator=g)
    scales = lambda n: torch.rand(n, device="cuda", generator=g) * 0.05 + 1e-4
    return codes(T, d_in), scales(T), codes(d_out, d_in), scales(d_out), \
        torch.randn(d_out, device="cuda", generator=g) * 20.0


def _sums(xq, wq):
    """The exact sums: integers below 2^53, in fp64."""
    w = wq.double().t()
    return torch.cat([xq[i:i + 1024].double() @ w for i in range(0, xq.shape[0], 1024)])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_every_form_against_the_exact_sums(shape):
    T, d_out, d_in = shape
    xq, sx, wq, sw, bias = _operands(*shape)
    acc = _sums(xq, wq)
    assert acc[0, 0] == (xq[0].long() * wq[0].long()).sum()
    assert acc[-1, -1] == (xq[-1].long() * wq[-1].long()).sum()
    f = acc.float() * sx[:, None] * sw[None, :]
    prod = (acc * sx.double()[:, None] * sw.double()[None, :])
    ref = prod + bias.double()[None, :]
    prod.abs_()
    for dt in (torch.bfloat16, torch.float32):
        # an output between guards
        whole = torch.full((T * d_out + 2048,), 77.0, dtype=dt, device="cuda")
        y = whole[1024:1024 + T * d_out].view(T, d_out)
        dora.dora_linear_i8(xq, sx, wq, sw, y=y)
        assert torch.equal(y, f.to(dt)), f"{dt}: bits"
        dora.dora_linear_i8(xq, sx, wq, sw, bias=bias, y=y)
        last = U if dt is torch.float32 else U + 2.0 ** -8
        tol = 2 * U * 1.01 * prod + last * 1.01 * (ref.abs() + 2 * U * prod)
        over = (y.double() - ref).abs() - tol
        assert not (over > 0).any() and not torch.isnan(over).any(), f"{dt}: {over.max()} over"
        assert (whole[:1024] == 77.0).all() and (whole[-1024:] == 77.0).all()
    assert dora.dora_get_device_status() == 0
