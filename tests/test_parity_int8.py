"""Parity of the 8-bit serving calls with the fp64 oracle.

Tolerances, from the arithmetic the header states (u = 2^-24, half an fp32
step, relative):
  * codes of dora_quantize_rows: 127/max|v| and its product with v are each
    rounded once, so the quotient is off by at most 2u relative, 127 * 2u of a
    code; a code is within 1/2 + 127 * 2u (1 + small) of the exact quotient.
  * codes of dora_rmsnorm_quant: h weight is rounded once more (in the value
    and in the maximum): 127 * 4u.
  * scale: max / 127 rounded once (u).  Behind the norm: the sum of squares,
    each thread's chain of n terms and the tree over at most 512 threads (10
    levels), is off by (n + 10) u, halved by the square root; its mean, the
    sum with eps (both halved), the root, the reciprocal, h weight, max / 127
    and the product add 6 u; n is at most 32, or the row over 512 threads
    where that is more.
  * y: the conversion and the first product are rounded (2u of the product
    term), the last operation once (u of y, or half a bf16 step, 2^-8).
  * h = x + residual: one rounding to the dtype.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import dora_adapter_factored_b200 as dora
import oracle
from dora_adapter_factored_b200 import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().cpu().double().numpy()


def _rand(T, d, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g) * scale
    x[:, ::17] *= 9.0
    return x.to(DTYPES[dt]).cuda()


def _check_codes(q, exact_u, slack, what):
    q = q.cpu().numpy().astype(np.float64)
    off = np.abs(q - exact_u)
    assert off.max(initial=0.0) <= 0.5 + slack, f"{what}: code off by {off.max()}"
    assert np.abs(q).max(initial=0.0) <= 127


def _check_rel(got, ref, tol, what):
    got, ref = _np(got), np.asarray(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    ok = ~np.isnan(ref)
    err = np.abs(got[ok] - ref[ok]) - tol * np.abs(ref[ok])
    assert err.max(initial=0.0) <= 0.0, f"{what}: beyond {tol} relative by {err.max()}"


def _check_quant(x, q, scale, what):
    _, s_ref, u_ref = oracle.quantize_rows(_np(x))
    _check_codes(q, u_ref, 127 * 2 * U * 1.01, what)
    _check_rel(scale, s_ref, U * 1.01, what)


def _check_norm(x, weight, residual, q, scale, h, what):
    hx = x
    if residual is not None:
        exact = _np(x) + _np(residual)
        half = torch.finfo(x.dtype).eps / 2
        # (the sum itself may be inexact in fp32 before the bf16 rounding)
        assert (np.abs(_np(h) - exact) <= (half + U) * np.abs(exact)).all(), what
        hx = h
    else:
        assert h is None
    v = oracle.rmsnorm(_np(hx), _np(weight), EPS)
    _, s_ref, u_ref = oracle.quantize_rows(v)
    d = x.shape[1]
    n = max(32, -(-d // 512) + 8)
    _check_codes(q, u_ref, 127 * 4 * U * 1.01, what)
    _check_rel(scale, s_ref, ((n + 12) / 2 + 6) * U, what)


WIDTHS = [1, 7, 8, 31, 33, 64, 255, 1000, 1024, 1032, 4096, 4099, 5120, 8192, 8200, 8201, 16384,
          16392, 40000]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_quantize_rows(d, dt):
    for T in (1, 2, 9):
        x = _rand(T, d, dt, 100 * d + T, 0.02)
        q, scale = dora.dora_quantize_rows(x)
        _check_quant(x, q, scale, f"{T}x{d} {dt}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_rmsnorm_quant(d, dt):
    for T, res in ((1, True), (2, False), (9, True)):
        x = _rand(T, d, dt, 7 * d + T)
        r = _rand(T, d, dt, 11 * d + T, 3.0) if res else None
        w = (1 + 0.2 * _rand(1, d, dt, 13 * d)[0].float()).to(DTYPES[dt])
        q, scale, h = dora.dora_rmsnorm_quant(x, w, EPS, residual=r)
        _check_norm(x, w, r, q, scale, h, f"{T}x{d} {dt} residual={res}")


@pytest.mark.parametrize("T,d,dt", [(2500, 64, "bf16"), (700, 1000, "f32"), (3001, 33, "bf16"),
                                    (1300, 2048, "bf16"), (500, 17000, "bf16")])
def test_many_rows(T, d, dt):
    """More rows than the grid has blocks: blocks walk rows."""
    x, r = _rand(T, d, dt, 3), _rand(T, d, dt, 4)
    w = _rand(1, d, dt, 5)[0].contiguous()
    q, scale = dora.dora_quantize_rows(x)
    _check_quant(x, q, scale, "quantize")
    q, scale, h = dora.dora_rmsnorm_quant(x, w, EPS, residual=r)
    _check_norm(x, w, r, q, scale, h, "norm")


@pytest.mark.parametrize("T,d,dt", [(20001, 3, "f32"), (20001, 7, "bf16"), (3001, 129, "f32"),
                                    (2503, 257, "bf16"), (1300, 1023, "bf16"), (700, 4099, "f32"),
                                    (650, 8191, "bf16"), (330, 8191, "f32"), (200, 16383, "f32"),
                                    (310, 16383, "bf16")])
def test_many_ragged_rows(T, d, dt):
    """Rows that start anywhere in a vector, more than the grid has blocks: the
    walked rows start alike, and no row sees its neighbours' elements."""
    x, r = _rand(T, d, dt, 3), _rand(T, d, dt, 4)
    w = (1 + 0.2 * _rand(1, d, dt, 5)[0].float()).to(DTYPES[dt]).contiguous()
    q, scale = dora.dora_quantize_rows(x)
    _check_quant(x, q, scale, "quantize")
    q, scale, h = dora.dora_rmsnorm_quant(x, w, EPS)
    _check_norm(x, w, None, q, scale, h, "norm")
    alone = (q, scale)
    q, scale, h = dora.dora_rmsnorm_quant(x, w, EPS, residual=r)
    _check_norm(x, w, r, q, scale, h, "norm of a sum")
    # every other row not finite: the rows between them keep their bits
    x[1::2] = float("nan")
    q, scale, _ = dora.dora_rmsnorm_quant(x, w, EPS)
    assert torch.equal(q[::2], alone[0][::2]) and torch.equal(scale[::2], alone[1][::2])
    assert not q[1::2].any() and torch.isnan(scale[1::2]).all()


@pytest.mark.parametrize("d", [1000, 40000])
def test_alignment_does_not_change_results(d):
    """Views that start off a 16-byte boundary take the element path: the same
    codes and h bit for bit; the norm's scale up to the order of its sum."""
    for dt in DTYPES.values():
        base = torch.randn(3 * d + 8, device="cuda").to(dt)
        rbase = torch.randn(3 * d + 8, device="cuda").to(dt)
        w = torch.randn(d, device="cuda").to(dt)
        x0, r0 = base[1:1 + 3 * d].view(3, d), rbase[3:3 + 3 * d].view(3, d)
        q0, s0 = dora.dora_quantize_rows(x0)
        q1, s1 = dora.dora_quantize_rows(x0.clone())
        assert torch.equal(q0, q1) and torch.equal(s0, s1)
        q0, s0, h0 = dora.dora_rmsnorm_quant(x0, w, EPS, residual=r0)
        q1, s1, h1 = dora.dora_rmsnorm_quant(x0.clone(), w, EPS, residual=r0.clone())
        assert torch.equal(q0, q1) and torch.equal(h0, h1)
        n = max(32, -(-d // 512) + 8)
        _check_rel(s0, _np(s1), (n + 12) * U, "scale")


@pytest.mark.parametrize("d", [64, 1024, 1001, 40000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_without_a_step(d, dt):
    """Zero rows, rows whose step is not a normal number, and rows with an
    infinity or a NaN do not touch their neighbours."""
    x = _rand(9, d, dt, 17)
    x[1] = 0.0
    x[2, d // 2] = float("inf")
    x[3, 0] = float("nan")
    x[4, d - 1] = float("-inf")
    x[5] = 1e-37   # a step below 2^-126
    x[6, 1:] = 0.0
    x[7] = float("nan")
    q, scale = dora.dora_quantize_rows(x)
    _check_quant(x, q, scale, "quantize")
    s = _np(scale)
    assert s[1] == 0 and s[5] == 0 and np.isnan(s[[2, 3, 4, 7]]).all()
    assert not q[[1, 2, 3, 4, 5, 7]].any()
    assert abs(int(q[6, 0])) == 127
    w = torch.ones(d, device="cuda", dtype=DTYPES[dt])
    x[5] = 0.0
    q, scale, _ = dora.dora_rmsnorm_quant(x, w, EPS)
    _check_norm(x, w, None, q, scale, None, "norm")
    s = _np(scale)
    assert s[1] == 0 and np.isnan(s[[2, 3, 4, 7]]).all() and not q[[1, 2, 3, 4, 5, 7]].any()
    # an infinity in the weight leaves no row finite; one in the residual only its own
    w2 = w.clone()
    w2[3] = float("inf")
    q, scale, _ = dora.dora_rmsnorm_quant(_rand(2, d, dt, 3), w2, EPS)
    assert torch.isnan(scale).all() and not q.any()
    r = _rand(2, d, dt, 4)
    r[1, 5] = float("nan")
    q, scale, h = dora.dora_rmsnorm_quant(_rand(2, d, dt, 3), w, EPS, residual=r)
    assert torch.isfinite(scale[0]) and torch.isnan(scale[1]) and q[0].any() and not q[1].any()


def test_sum_of_squares_out_of_range_is_not_finite():
    x = torch.full((1, 64), 1e30, device="cuda")
    q, scale, _ = dora.dora_rmsnorm_quant(x, torch.ones(64, device="cuda"), EPS)
    assert torch.isnan(scale).all() and not q.any()


def test_halves_go_to_even():
    x = torch.zeros(1, 64, device="cuda")
    x[0, 0] = 127.0
    x[0, 1:8] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 3.5, 126.5])
    q, scale = dora.dora_quantize_rows(x)
    assert scale.item() == 1.0
    assert q[0, :8].tolist() == [127, 0, 2, 2, 0, -2, 4, 126]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (2, 64), (5, 1000), (9, 1001), (700, 264),
                                 (2500, 33), (41, 40000), (1, 8192)])
def test_dequantize_rows(T, d, dt):
    """One fp32 product, and for bf16 its rounding: bit for bit."""
    q, scale = _codes(T, d, T + d), _scales(T, d)
    if T > 2:
        scale[1], scale[2] = float("nan"), 0.0
    want = (q.cpu().float() * scale.cpu()[:, None]).to(DTYPES[dt])
    x = dora.dora_dequantize_rows(q, scale, DTYPES[dt])
    assert torch.equal(torch.isnan(x.cpu()), torch.isnan(want))
    assert torch.equal(x.cpu().nan_to_num(), want.nan_to_num())
    # operands and result off their boundaries
    qb = torch.empty(T * d + 3, dtype=torch.int8, device="cuda")[3:].view(T, d).copy_(q)
    xb, xw, xg = _guarded(T * d + 1, DTYPES[dt])
    out = dora.dora_dequantize_rows(qb, scale, x=xb[1:].view(T, d))
    _intact((xw, xg))
    assert torch.equal(out.nan_to_num(), x.nan_to_num())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(30011, 1401), (300007, 137), (6000001, 7), (20000003, 2)])
def test_dequantize_more_than_the_grid_at_once(T, d, dt):
    """Threads that follow their rows from one vector to the next, over vectors
    of one row, of two and of several."""
    g = torch.Generator("cuda").manual_seed(d)
    q = torch.randint(-127, 128, (T, d), dtype=torch.int8, device="cuda", generator=g)
    scale = torch.rand(T, device="cuda", generator=g) + 0.5
    want = (q.float() * scale[:, None]).to(DTYPES[dt])
    assert torch.equal(dora.dora_dequantize_rows(q, scale, DTYPES[dt]), want)


def test_weight_held_as_codes_through_norm_and_merge():
    """A quantised base weight, dequantised for the calls that read bf16."""
    W0 = _rand(96, 256, "bf16", 1, 0.02)
    A, B = _rand(16, 256, "bf16", 2, 0.03), _rand(96, 16, "bf16", 3, 0.02)
    q, scale = dora.dora_quantize_rows(W0)
    W = dora.dora_dequantize_rows(q, scale)
    n, _ = dora.dora_factored_norm(W, A, B, 2.0)
    ref = oracle.dense_row_norm(_np(W), _np(A), _np(B), 2.0)
    assert np.max(np.abs(_np(n) - ref) / ref) < 1e-3
    half = 0.5 + 127 * 2 * U + 1e-4  # half a step of each row, and bf16's rounding
    assert (np.abs(_np(W) - _np(W0)) <= half * _np(scale)[:, None] + 2.0 ** -8 * np.abs(_np(W0))
            + 2.0 ** -8 * _np(scale)[:, None]).all()


@pytest.mark.parametrize("over", ["x", "residual"])
@pytest.mark.parametrize("d", [1024, 999, 40000])
def test_h_in_place(over, d):
    x, r = _rand(5, d, "bf16", 1), _rand(5, d, "bf16", 2)
    w = _rand(1, d, "bf16", 3)[0].contiguous()
    q0, s0, h0 = dora.dora_rmsnorm_quant(x, w, EPS, residual=r)
    x1, r1 = x.clone(), r.clone()
    out = x1 if over == "x" else r1
    q1, s1, h1 = dora.dora_rmsnorm_quant(x1, w, EPS, residual=r1, h_out=out)
    assert h1.data_ptr() == out.data_ptr()
    assert torch.equal(q0, q1) and torch.equal(s0, s1) and torch.equal(h0, h1)
    assert torch.equal(r1 if over == "x" else x1, r if over == "x" else x)


# ------------------------------------------------------------------ linear

def _codes(rows, cols, seed, low=-128):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, 128, (rows, cols), generator=g).to(torch.int8).cuda()


def _scales(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(n, generator=g) * 0.05 + 1e-4).cuda()


def _check_linear(y, xq, sx, wq, sw, bias, what):
    acc, ref = oracle.linear_i8(_np(xq), _np(sx), _np(wq), _np(sw),
                                None if bias is None else _np(bias))
    prod = np.abs(acc * _np(sx)[:, None] * _np(sw)[None, :])
    last = U if y.dtype == torch.float32 else U + 2.0 ** -8
    err = np.abs(_np(y) - ref)
    tol = 2 * U * 1.01 * prod + last * 1.01 * (np.abs(ref) + 2 * U * prod)
    assert (err <= tol).all(), f"{what}: {np.max(err - tol)} over"
    if bias is None:  # the stated operations, bit for bit
        f = acc.astype(np.float32) * sx.cpu().numpy()[:, None] * sw.cpu().numpy()[None, :]
        assert torch.equal(y.cpu(), torch.from_numpy(f).to(y.dtype)), f"{what}: bits"


TOKENS = [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 77, 128, 129, 200, 256, 257, 300, 520, 700]
LAYERS = [(1, 16), (7, 1), (100, 15), (128, 128), (129, 144), (1000, 1003), (264, 4096),
          (1024, 1040), (33, 2064)]


@pytest.mark.parametrize("d_out,d_in", LAYERS)
def test_linear_i8(d_out, d_in):
    wq, sw = _codes(d_out, d_in, d_out + d_in), _scales(d_out, 1)
    xq, sx = _codes(max(TOKENS), d_in, 5), _scales(max(TOKENS), 2)
    bias = torch.randn(d_out, generator=torch.Generator().manual_seed(3)).cuda()
    for i, T in enumerate(TOKENS):
        dt = torch.float32 if i % 2 else torch.bfloat16
        b = bias if i % 3 == 0 else None
        y = dora.dora_linear_i8(xq[:T], sx[:T], wq, sw, bias=b, dtype=dt)
        torch.cuda.synchronize()
        assert dora.dora_get_device_status() == 0
        _check_linear(y, xq[:T], sx[:T], wq, sw, b, f"T={T} {d_out}x{d_in}")


@pytest.mark.parametrize("T", [1, 3, 20, 300])
def test_linear_long_k_extreme_codes(T):
    """The largest sum: every product 128 * 128 over the longest k."""
    d_in = dora.DORA_MAX_I8_K
    xq = torch.full((T, d_in), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((3, d_in), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    sx, sw = torch.ones(T, device="cuda"), torch.ones(3, device="cuda")
    y = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
    want = np.float32([128 * 128 * d_in, -128 * 127 * d_in, 128 * 128 * d_in])
    assert (y.cpu().numpy() == want[None, :]).all()


@pytest.mark.parametrize("d_out,d_in", [(520, 1024), (300, 1003), (4096, 512)])
def test_a_token_does_not_depend_on_its_batch(d_out, d_in):
    wq, sw = _codes(d_out, d_in, 1), _scales(d_out, 1)
    xq, sx = _codes(600, d_in, 2), _scales(600, 2)
    bias = torch.randn(d_out, device="cuda")
    whole = dora.dora_linear_i8(xq, sx, wq, sw, bias=bias)
    for T in (1, 2, 5, 9, 40, 130, 300):
        part = dora.dora_linear_i8(xq[:T], sx[:T], wq, sw, bias=bias)
        assert torch.equal(part, whole[:T]), T


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_linear_unaligned_operands(T):
    """Operands that start at any byte."""
    d_out, d_in = 200, 512
    xb, wb = _codes(1, T * d_in + 16, 1)[0], _codes(1, d_out * d_in + 16, 2)[0]
    xq, wq = xb[3:3 + T * d_in].view(T, d_in), wb[5:5 + d_out * d_in].view(d_out, d_in)
    sx, sw = _scales(T, 1), _scales(d_out, 2)
    y = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
    _check_linear(y, xq, sx, wq, sw, None, f"T={T}")
    yb = torch.empty(T * d_out + 1, dtype=torch.bfloat16, device="cuda")
    out = dora.dora_linear_i8(xq.clone(), sx, wq.clone(), sw, y=yb[1:].view(T, d_out))
    _check_linear(out, xq, sx, wq, sw, None, f"T={T}, y off its boundary")


def test_scale_nan_and_zero_reach_only_their_own_outputs():
    for T in (2, 40, 300):
        wq, sw = _codes(96, 256, 1), _scales(96, 1)
        xq, sx = _codes(T, 256, 2), _scales(T, 2)
        sx[1], sx[0] = float("nan"), 0.0
        sw[5] = float("nan")
        y = dora.dora_linear_i8(xq, sx, wq, sw)
        bad = torch.isnan(y)
        assert bad[1].all() and bad[:, 5].all()
        bad[1] = False
        bad[:, 5] = False
        assert not bad.any()
        keep = [j for j in range(96) if j != 5]
        assert not y[0, keep].any()


# ------------------------------------------------- empties, guards, streams

def test_no_rows():
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    before = dora.dora_launch_count()
    q, s = dora.dora_quantize_rows(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    q, s, h = dora.dora_rmsnorm_quant(x, w, EPS, residual=x.clone())
    assert h.shape == (0, 64)
    assert dora.dora_dequantize_rows(q, s).shape == (0, 64)
    y = dora.dora_linear_i8(q, s, _codes(8, 64, 1), _scales(8, 1))
    assert y.shape == (0, 8)
    assert dora.dora_launch_count() == before


def _guarded(n, dtype, guard=4096):
    size = torch.empty(0, dtype=dtype).element_size()
    whole = torch.full(((n + 2 * guard) * size,), 0x5A, dtype=torch.uint8, device="cuda")
    return whole.view(dtype)[guard:guard + n], whole, guard * size


def _intact(*guards):
    torch.cuda.synchronize()
    for whole, g in guards:
        assert bool((whole[:g] == 0x5A).all()) and bool((whole[-g:] == 0x5A).all())


@pytest.mark.parametrize("T,d,d_out", [(3, 1003, 130), (17, 1024, 1001), (131, 272, 300),
                                       (300, 640, 520), (140, 1001, 77)])
def test_nothing_is_written_outside_the_outputs(T, d, d_out):
    x, r, w = _rand(T, d, "bf16", 1), _rand(T, d, "bf16", 2), _rand(1, d, "bf16", 3)[0].contiguous()
    q, qw, qg = _guarded(T * d, torch.int8)
    s, sw_, sg = _guarded(T, torch.float32)
    h, hw, hg = _guarded(T * d, torch.bfloat16)
    dora.dora_rmsnorm_quant(x, w, EPS, residual=r, h_out=h.view(T, d), q=q.view(T, d), scale=s)
    dora.dora_quantize_rows(x, q=q.view(T, d), scale=s)
    need = dora.dora_linear_i8_workspace_size(T, d_out, d)
    wsw = torch.full((need + 8192 + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    off = 4096 + (-(wsw.data_ptr() + 4096)) % 256
    for dt in (torch.bfloat16, torch.float32):
        y, yw, yg = _guarded(T * d_out, dt)
        dora.dora_linear_i8(q.view(T, d), s, _codes(d_out, d, 4), _scales(d_out, 5),
                            y=y.view(T, d_out), ws=wsw[off:off + need])
        _intact((yw, yg))
    _intact((qw, qg), (sw_, sg), (hw, hg))
    assert bool((wsw[:off] == 0x5A).all()) and bool((wsw[off + need:] == 0x5A).all())
    assert dora.dora_get_device_status() == 0


def _layer(x, r, w, wq, sw, bias, stream=None):
    q, s, h = dora.dora_rmsnorm_quant(x, w, EPS, residual=r, stream=stream)
    y = dora.dora_linear_i8(q, s, wq, sw, bias=bias, stream=stream)
    q2, s2 = dora.dora_quantize_rows(y, stream=stream)
    return h, q, s, y, q2, s2, dora.dora_dequantize_rows(q2, s2, stream=stream)


@pytest.mark.parametrize("T", [1, 24, 150, 600])
def test_streams_and_graphs(T):
    """The layer on side streams, two at once, and captured and replayed on
    new inputs: the bits of the plain call."""
    d, d_out = 1024, 1536
    x, r, w = _rand(T, d, "bf16", 1), _rand(T, d, "bf16", 2), _rand(1, d, "bf16", 3)[0].contiguous()
    wq, sw, bias = _codes(d_out, d, 4), _scales(d_out, 5), torch.randn(d_out, device="cuda")
    ref = _layer(x, r, w, wq, sw, bias)
    ref2 = _layer(r, x, w, wq, sw, bias)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = _layer(x, r, w, wq, sw, bias, stream=a)
        got2 = _layer(r, x, w, wq, sw, bias, stream=b.cuda_stream)
    torch.cuda.synchronize()
    for k in range(7):
        assert torch.equal(ref[k], got[k]) and torch.equal(ref2[k], got2[k])
    xs, rs = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(xs, rs, w, wq, sw, bias)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(ref, out))
    xs.copy_(r)
    rs.copy_(x)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(ref2, out))
    assert dora.dora_get_device_status() == 0


# A fresh process whose first calls happen inside a stream capture: the one-time
# setup of the kernels then runs during the capture.
_FIRST_CALL_IN_CAPTURE = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import dora_adapter_factored_b200 as dora
g = torch.Generator().manual_seed(5)
w = torch.ones(512, device="cuda").bfloat16()
wq = torch.randint(-127, 128, (384, 512), generator=g).to(torch.int8).cuda()
sw = torch.rand(384, generator=g).cuda()
outs = []
for T in (3, 40, 300):
    x = torch.randn(T, 512, generator=g).bfloat16().cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s, h = dora.dora_rmsnorm_quant(x, w, 1e-6, residual=x)
        y = dora.dora_linear_i8(q, s, wq, sw)
        z = dora.dora_dequantize_rows(*dora.dora_quantize_rows(y))
    graph.replay()
    torch.cuda.synchronize()
    outs.append((x, q, s, h, y, z))
for x, *got in outs:
    q, s, h = dora.dora_rmsnorm_quant(x, w, 1e-6, residual=x)
    y = dora.dora_linear_i8(q, s, wq, sw)
    for a, b in zip(got, (q, s, h, y, dora.dora_dequantize_rows(*dora.dora_quantize_rows(y)))):
        assert torch.equal(a, b)
assert dora.dora_get_device_status() == 0
print("OK")
"""


def _child(code, *args):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code, root, *args], capture_output=True, text=True,
                         timeout=600)
    assert res.returncode == 0 and "OK" in res.stdout, res.stdout + res.stderr


def test_first_calls_inside_a_capture():
    _child(_FIRST_CALL_IN_CAPTURE)


# The debug build on odd shapes: bounds-checked stores, the release build's bits.
_DEBUG_BUILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import dora_adapter_factored_b200 as dora
from dora_adapter_factored_b200 import build
dora.load_library(build.library_path(debug=sys.argv[2] == "debug"))
g = torch.Generator().manual_seed(7)
out = []
for T, d, d_out in ((1, 7, 5), (3, 1003, 130), (9, 264, 1001), (40, 520, 264), (140, 1001, 77),
                    (300, 4104, 520), (600, 144, 300), (2, 40000, 9)):
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(T, d, generator=g).to(dt).cuda()
        w = torch.randn(d, generator=g).to(dt).cuda()
        q, s, h = dora.dora_rmsnorm_quant(x, w, 1e-6, residual=x)
        q2, s2 = dora.dora_quantize_rows(h)
        wq = torch.randint(-128, 128, (d_out, d), generator=g).to(torch.int8).cuda()
        sw = torch.rand(d_out, generator=g).cuda()
        y = dora.dora_linear_i8(q, s, wq, sw, bias=sw, dtype=dt)
        out += [q, s, h, q2, s2, y, dora.dora_dequantize_rows(q, s, dt)]
torch.cuda.synchronize()
assert dora.dora_get_device_status() == 0
torch.save([t.cpu() for t in out], sys.argv[3])
print("OK")
"""


def test_debug_build_gives_the_same_bits(built_library, built_debug_library, tmp_path):
    for kind in ("debug", "release"):
        _child(_DEBUG_BUILD, kind, str(tmp_path / kind))
    a, b = (torch.load(tmp_path / kind) for kind in ("debug", "release"))
    assert len(a) == len(b) and all(torch.equal(u, v) for u, v in zip(a, b))


def test_linear_gives_up_on_a_wait_that_runs_out():
    """With a limit of 1 ns the pipelines' waits run out: the status says so, the
    context stays usable, and the next call is right."""
    wq, sw = _codes(1024, 4096, 1), _scales(1024, 1)
    xq, sx = _codes(600, 4096, 2), _scales(600, 2)
    for T in (40, 600):
        ref = dora.dora_linear_i8(xq[:T], sx[:T], wq, sw)
        assert dora.dora_get_device_status() == 0
        dora.dora_set_wait_timeout_ns(1)
        try:
            dora.dora_linear_i8(xq[:T], sx[:T], wq, sw)
            status = dora.dora_get_device_status()
        finally:
            dora.dora_set_wait_timeout_ns(0)
        assert status in (0, 5)
        got = dora.dora_linear_i8(xq[:T], sx[:T], wq, sw)
        assert dora.dora_get_device_status() == 0 and torch.equal(got, ref)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows are where they belong."""
    rows, cols = 131200, 16392
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    last = _rand(3, cols, "bf16", 1)
    x[-3:] = last
    q, scale = dora.dora_quantize_rows(x)
    _check_quant(last, q[-3:], scale[-3:], "last rows")
    assert not scale[:-3].any() and not q[:-3:1000].any()
    w = torch.ones(cols, device="cuda", dtype=torch.bfloat16)
    q, scale, h = dora.dora_rmsnorm_quant(x, w, EPS, residual=x, h_out=x, q=q, scale=scale)
    _check_norm(last, w, last, q[-3:], scale[-3:], h[-3:], "norm of last rows")
    del x, h
    v = dora.dora_dequantize_rows(q, scale)
    want = (q[-3:].cpu().float() * scale[-3:].cpu()[:, None]).bfloat16()
    assert torch.equal(v[-3:].cpu(), want)
    del v, q, scale
    T, d_out, d_in = 70000, 32776, 48
    xq, sx = _codes(T, d_in, 3), _scales(T, 3)
    wq, sw = _codes(d_out, d_in, 4), _scales(d_out, 4)
    y = dora.dora_linear_i8(xq, sx, wq, sw)
    for rows in (slice(0, 2), slice(T // 2, T // 2 + 2), slice(T - 2, T)):
        _check_linear(y[rows], xq[rows], sx[rows], wq, sw, None, f"rows {rows}")
    assert dora.dora_get_device_status() == 0


def test_refusals():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(4, 64, device="cuda", dtype=torch.int8)
    s = torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        dora.dora_quantize_rows(x.t())
    with pytest.raises(ValueError, match="two dimensions"):
        dora.dora_quantize_rows(w)
    with pytest.raises(TypeError, match="dtype"):
        dora.dora_quantize_rows(x.half())
    with pytest.raises(TypeError, match="scale must be"):
        dora.dora_quantize_rows(x, scale=s.half())
    with pytest.raises(ValueError, match="shape"):
        dora.dora_quantize_rows(x, q=q[:2])
    with pytest.raises(TypeError, match="weight must be"):
        dora.dora_rmsnorm_quant(x, w.float(), EPS)
    with pytest.raises(ValueError, match="residual"):
        dora.dora_rmsnorm_quant(x, w, EPS, h_out=x)
    with pytest.raises(ValueError, match="residual must be on"):
        dora.dora_rmsnorm_quant(x, w, EPS, residual=x.cpu())
    with pytest.raises(dora.DoraError):
        dora.dora_rmsnorm_quant(x, w, 0.0)
    with pytest.raises(dora.DoraError):
        dora.dora_rmsnorm_quant(x, w, EPS, residual=x.clone(), h_out=w.new_zeros(4, 64),
                                q=q, scale=x.view(-1).view(torch.float32)[:4])
    with pytest.raises(TypeError, match="dtype"):
        dora.dora_dequantize_rows(q, s, torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        dora.dora_dequantize_rows(q.t(), torch.ones(64, device="cuda"))
    with pytest.raises(ValueError, match="x must have shape"):
        dora.dora_dequantize_rows(q, s, x=x[:2])
    with pytest.raises(TypeError, match="xq must be"):
        dora.dora_linear_i8(x, s, q, s)
    with pytest.raises(ValueError, match="wq must have shape"):
        dora.dora_linear_i8(q, s, q[:, :32].contiguous(), s)
    with pytest.raises(ValueError, match="x_scale must have shape"):
        dora.dora_linear_i8(q, s[:3], q, s)
    with pytest.raises(TypeError, match="dtype"):
        dora.dora_linear_i8(q, s, q, s, dtype=torch.float16)
    with pytest.raises(ValueError, match="bias must be on"):
        dora.dora_linear_i8(q, s, q, s, bias=torch.zeros(4))
    assert dora.dora_get_device_status() == 0


# ------------------------------------------------------- the set in use

@pytest.mark.parametrize("T", [1, 19, 300])
def test_merged_module_served_in_8_bits(T):
    """Factored norm, merge and row quantisation once; norm and linear per
    step.  The codes' own errors bound the distance to the fp64 module: each
    operand is off by at most half a step (and the roundings of its fp32
    quotient), so |dy_tj| <= sum_k |v_tk| sw_j/2 + |W_jk| sx_t/2 + sx_t sw_j/4."""
    d_out, d_in, r, s, eps = 520, 768, 64, 2.0, 2.0 ** -7
    g = torch.Generator().manual_seed(5)
    W0 = (0.02 * torch.randn(d_out, d_in, generator=g)).bfloat16().cuda()
    A = ((torch.rand(r, d_in, generator=g) * 2 - 1) / d_in ** 0.5).bfloat16().cuda()
    B = (0.02 * torch.randn(d_out, r, generator=g)).bfloat16().cuda()
    n, _ = dora.dora_factored_norm(W0, A, B, s)
    m = n * (1 + 0.005 * torch.randn(d_out, generator=g).cuda())
    W = dora.dora_merge_weight(W0, A, B, m, n, s, eps)
    wq, sw = dora.dora_quantize_rows(W)
    x, res = _rand(T, d_in, "bf16", 6), _rand(T, d_in, "bf16", 7, 3.0)
    weight = (1 + 0.1 * torch.randn(d_in, generator=g)).bfloat16().cuda()
    xq, sx, h = dora.dora_rmsnorm_quant(x, weight, EPS, residual=res)
    y = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
    torch.cuda.synchronize()
    assert dora.dora_get_device_status() == 0
    _check_quant(W, wq, sw, "W'")
    _check_norm(x, weight, res, xq, sx, h, "h")
    _check_linear(y, xq, sx, wq, sw, None, "y")
    v, Wn = oracle.rmsnorm(_np(h), _np(weight), EPS), _np(W)
    ref = v @ Wn.T
    half = 0.5 + 127 * 4 * U + 1e-4  # half a step, the quotient's roundings, the scale's
    bound = half * (np.abs(v).sum(1)[:, None] * _np(sw) + _np(sx)[:, None] * np.abs(Wn).sum(1)) \
        + half * half * d_in * _np(sx)[:, None] * _np(sw)
    assert (np.abs(_np(y) - ref) <= bound).all()
    # and the codes are worth having: 8 bits on both sides keep y to a few percent
    assert np.linalg.norm(_np(y) - ref) <= 0.05 * np.linalg.norm(ref)
