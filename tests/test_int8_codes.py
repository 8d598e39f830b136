"""The codes of rows against the definition itself, q = round(127 v / max|v|) half
to even, where they are decided by the last bit: values half-way between two
codes, which the tolerances of the parity tests leave open.

No tolerance: for bf16 values 127 v is exact in fp64 (15 bits) and its quotient
by max|v| is rounded once, to a half only where it is one (any other quotient of
8-bit mantissas is at least 2^-10 of its size from a half)."""
import numpy as np
import pytest
import torch

import dora_adapter_factored_b200 as dora

pytestmark = pytest.mark.gpu


def _every_mantissa(d):
    """[128, d] bf16: row i has the maximum 128 + i (in units of 2^-9) and, in
    turn, every value of eight mantissa bits at or below it, both signs, down to
    2^-11 of it."""
    v = np.concatenate([np.arange(128, 256) * 2.0 ** -s for s in range(12)])
    x = np.zeros((128, d))
    for i in range(128):
        top = 128.0 + i
        own = v[v <= top]
        own = np.concatenate([[top, -top, top / 2, -top / 2], own, -own])
        x[i] = np.resize(own, d)
        x[i, d - 1] = top / 2  # a ragged row's loose elements too
    return torch.from_numpy(x * 2.0 ** -9).to(torch.bfloat16)


def _definition(x):
    v = x.double().numpy()
    return np.rint(127 * v / np.abs(v).max(axis=1, keepdims=True))


@pytest.mark.parametrize("d", [256, 1001, 2999, 4096, 40000])
def test_codes_of_bf16_rows_are_the_definitions(d):
    x = _every_mantissa(d)
    want = _definition(x)
    xc = x.cuda()
    q, scale = dora.dora_quantize_rows(xc)
    assert np.array_equal(q.cpu().numpy(), want)
    top = x.float().abs().amax(dim=1)
    assert torch.equal(scale.cpu(), top / 127.0)
    # held in fp32, and off its boundary
    q, _ = dora.dora_quantize_rows(xc.float())
    assert np.array_equal(q.cpu().numpy(), want)
    off = torch.empty(x.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(x.shape)
    q, _ = dora.dora_quantize_rows(off.copy_(xc))
    assert np.array_equal(q.cpu().numpy(), want)
    # behind the norm with a weight of powers of two: the rms is common to the row
    w = torch.full((d,), 0.5, dtype=torch.bfloat16, device="cuda")
    q, _, _ = dora.dora_rmsnorm_quant(xc, w, 1e-6)
    assert np.array_equal(q.cpu().numpy(), want)
    q, _, h = dora.dora_rmsnorm_quant(xc, w, 1e-6, residual=torch.zeros_like(xc))
    assert torch.equal(h, xc) and np.array_equal(q.cpu().numpy(), want)


def test_a_half_of_the_largest_fp32_value_goes_to_64():
    g = torch.Generator().manual_seed(3)
    x = torch.zeros(4096, 64)
    x[:, 0] = torch.rand(4096, generator=g) + 1.0
    x[:, 1], x[:, 2] = x[:, 0] / 2, -x[:, 0] / 2
    q, _ = dora.dora_quantize_rows(x.cuda())
    assert (q[:, 0] == 127).all() and (q[:, 1] == 64).all() and (q[:, 2] == -64).all()
    assert not q[:, 3:].any()
