"""The norm's rows whose step is, or may be, no normal number: the rule is about
v = h w / rms, so neither h w below fp32's normal numbers nor a large rms
decides it.  Against the fp64 oracle, with the tolerances derived in
test_parity_int8.py (lifting a row by a power of two rounds nothing); whether a
row has a step is decided by the oracle, and every row here is at least 1 %
from the border."""
import numpy as np
import pytest
import torch

import dora_adapter_factored_b200 as dora
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# (weight's size, eps, sizes of the rows of h)
CASES = {
    "h below the step": (1.0, 1e-6, [1.0, 1e-37, 1e-35, 0.0, 1e-30, 3e-39, 1e3, 2e-38, 1e-40]),
    "weight below the step": (1e-37, 1e-6, [1.0, 1e3, 1e-3, 0.0, 3e4, 1e-20]),
    "products below fp32": (1e-25, 1e-30, [1e-25, 1e-24, 1e-10, 0.0, 1e-15, 1e-30, 1.0]),
    "products below the step": (1e-36, 1e-12, [1e-2, 1e-3, 1e-5, 1.0, 30.0, 1e-9]),
    "large weight": (1e35, 1e-6, [1.0, 1e-10, 1e-30, 20.0, 0.0]),
}


def _rows(sizes, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(len(sizes), d, generator=g, dtype=torch.float64).clamp(-4, 4)
    return (x * torch.tensor(sizes, dtype=torch.float64)[:, None]).to(DTYPES[dt]).cuda()


def _check(h, w, eps, q, scale, what):
    d = h.shape[1]
    v = oracle.rmsnorm(h.double().cpu().numpy(), w.double().cpu().numpy(), eps)
    _, s_ref, u_ref = oracle.quantize_rows(v)
    with np.errstate(divide="ignore"):
        edge = np.abs(np.abs(v).max(1) / 127 * 2.0 ** 126 - 1.0)
    assert (edge > 0.01).all(), "a row at the border: choose another"
    got = scale.double().cpu().numpy()
    assert ((got == 0) == (s_ref == 0)).all(), f"{what}: {got} against {s_ref}"
    n = max(32, -(-d // 512) + 8)
    assert (np.abs(got - s_ref) <= ((n + 12) / 2 + 6) * U * s_ref).all(), what
    off = np.abs(q.cpu().numpy() - u_ref)
    assert off.max() <= 0.5 + 127 * 4 * U * 1.01, f"{what}: code off by {off.max()}"
    assert not q[torch.from_numpy(s_ref == 0).cuda()].any()
    return s_ref


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [7, 64, 250, 1001, 1024, 4099, 5120, 17000, 40000, 40001])
def test_the_rule_is_about_the_normed_row(d, dt):
    for k, (what, (ws, eps, sizes)) in enumerate(CASES.items()):
        g = torch.Generator().manual_seed(d + k)
        w = ((1 + 0.2 * torch.randn(d, generator=g, dtype=torch.float64)) * ws).to(DTYPES[dt]).cuda()
        x = _rows(sizes, d, dt, 3 * d + k)
        q, scale, _ = dora.dora_rmsnorm_quant(x, w, eps)
        s_ref = _check(x, w, eps, q, scale, what)
        assert (s_ref != 0).any() == (what != "weight below the step")
        zero = torch.zeros_like(x)
        q2, scale2, h = dora.dora_rmsnorm_quant(x, w, eps, residual=zero)
        assert torch.equal(h, x)
        _check(h, w, eps, q2, scale2, what + ", with a residual")
        inplace = x.clone()
        q3, scale3, _ = dora.dora_rmsnorm_quant(inplace, w, eps, residual=zero, h_out=inplace)
        assert torch.equal(q3, q2) and torch.equal(scale3, scale2)
        off = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)
        q4, scale4, _ = dora.dora_rmsnorm_quant(off, w, eps)
        _check(off, w, eps, q4, scale4, what + ", off its boundary")
    assert dora.dora_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 1001, 8192, 20000])
def test_neighbours_of_such_rows_keep_their_bits(d):
    """More rows than the grid has blocks, every third one taken again."""
    T = 3000 if d < 5000 else 900
    x = torch.randn(T, d, device="cuda")
    w = 1 + 0.2 * torch.randn(d, device="cuda")
    q0, s0, _ = dora.dora_rmsnorm_quant(x, w, 1e-6)
    tiny = x[1::3] * 1e-37
    x[1::3] = tiny
    q, s, _ = dora.dora_rmsnorm_quant(x, w, 1e-6)
    keep = torch.arange(T, device="cuda") % 3 != 1
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    _check(tiny[-5:], w, 1e-6, q[1::3][-5:], s[1::3][-5:], "tiny rows")
    _check(tiny[:5], w, 1e-6, q[1::3][:5], s[1::3][:5], "tiny rows")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40000, 80000])
def test_a_scale_beyond_fp32_is_not_finite(d, dt):
    """Codes never stand for infinities: a row whose scale, or whose mean square
    with eps, leaves fp32's range is held like one that is not finite.  The first
    row's scale is 2^127 sqrt(d) / 127: 2.7e38 at 40000, 3.8e38 at 80000, where
    fp32 ends at 3.4e38."""
    x = torch.zeros(3, d)
    x[0, 7] = 0.125          # v = 2^127 sqrt(d) at one place
    x[1] = 0.125             # v = 2^127
    x[2, ::2] = -0.125
    x = x.to(DTYPES[dt]).cuda()
    w = torch.full((d,), 2.0 ** 127, dtype=DTYPES[dt], device="cuda")
    for residual in (None, torch.zeros_like(x)):
        q, scale, _ = dora.dora_rmsnorm_quant(x, w, 1e-30, residual=residual)
        v = oracle.rmsnorm(x.double().cpu().numpy(), w.double().cpu().numpy(), 1e-30)
        _, s_ref, _ = oracle.quantize_rows(v)
        first = 0 if d == 40000 else 1
        if first:
            assert torch.isnan(scale[0]) and not q[0].any()
        else:
            assert q[0, 7] == 127 and int(q[0].abs().sum()) == 127
        # a thread's chain of terms, ten levels and six more roundings
        tol = ((d / 512 + 8 + 12) / 2 + 6) * U
        assert (np.abs(scale.double().cpu().numpy() - s_ref) <= tol * s_ref)[first:].all()
        assert (q[1] == 127).all() and (q[2, ::2] == -127).all() and not q[2, 1::2].any()
    h = torch.full((1, 1), 1.5e19, dtype=DTYPES[dt], device="cuda")
    q, scale, _ = dora.dora_rmsnorm_quant(h, torch.ones_like(h[0]), 3e38)
    assert torch.isnan(scale).all() and not q.any()
