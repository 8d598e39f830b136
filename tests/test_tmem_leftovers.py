"""Calls that use tensor memory do not depend on what the kernel before them left
there: the int8 product leaves negative int32 sums, which as fp32 bits are NaN,
in all of its columns; a module with NaN or infinities leaves those."""
import numpy as np
import pytest
import torch

import dora_adapter_factored_b200 as dora
import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def poison():
    """Fills every column of every SM's tensor memory with fp32 NaN patterns: all
    sums are -16 = 0xfffffff0, two accumulators of 256 columns on every pair."""
    T, d_out, d_in = 8192, 8192, 16
    p = dora.dora_linear_i8_plan(T, d_out, d_in)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert p["kernel"] == 2 and p["tokens"] == 256
    assert p["token_tiles"] * p["channel_tiles"] >= 2 * (sms // 2)
    xq = torch.ones(T, d_in, dtype=torch.int8, device="cuda")
    wq = torch.full((d_out, d_in), -1, dtype=torch.int8, device="cuda")
    s, w = torch.ones(T, device="cuda"), torch.ones(d_out, device="cuda")
    y = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")

    def run():
        dora.dora_linear_i8(xq, s, wq, w, y=y)
    run()
    assert (y == -16.0).all()
    return run


def _module(d_out, d_in, r, seed):
    g = torch.Generator().manual_seed(seed)
    W0 = (0.02 * torch.randn(d_out, d_in, generator=g)).bfloat16()
    A = ((torch.rand(r, d_in, generator=g) * 2 - 1) / d_in ** 0.5).bfloat16()
    B = (0.02 * torch.randn(d_out, r, generator=g)).bfloat16()
    return W0, A, B


def _np(t):
    return t.double().cpu().numpy()


def _check(n, W0, A, B, s, what):
    ref = oracle.dense_row_norm(_np(W0), _np(A), _np(B), s)
    err = np.abs(_np(n) - ref) / ref
    assert not np.isnan(err).any() and err.max() <= 1e-3, f"{what}: {err.max()}"


RANKS = [8, 16, 24, 32, 40, 48, 72, 80, 104, 112, 136, 144, 168, 200, 208, 232, 240, 264, 272, 296,
         384, 392, 504, 512]


@pytest.mark.parametrize("r", RANKS)
def test_norm_behind_the_int8_product(poison, r):
    for d_out, d_in in ((300, 136), (2048, 1024)):
        W0, A, B = _module(d_out, d_in, r, r + d_out)
        Wc, Ac, Bc = W0.cuda(), A.cuda(), B.cuda()
        poison()
        n, _ = dora.dora_factored_norm(Wc, Ac, Bc, 2.0)
        _check(n, W0, A, B, 2.0, f"{d_out}x{d_in} r{r}")
        poison()
        sq = dora.dora_factored_norm_sq(Wc, Ac, Bc, 2.0)
        assert torch.equal(sq.sqrt(), n)
    assert dora.dora_get_device_status() == 0


def test_grouped_norm_behind_the_int8_product(poison):
    mods, ref = [], []
    for i, r in enumerate((16, 384, 48, 8, 80, 264, 40, 512, 112)):
        W0, A, B = _module(300 + 100 * i, 256, r, i)
        ref.append((W0, A, B))
        mods.append(dict(W0=W0.cuda(), A=A.cuda(), B=B.cuda(), s=1.5,
                         n_out=torch.empty(300 + 100 * i, device="cuda")))
    poison()
    dora.dora_factored_norm_grouped(mods)
    for m, (W0, A, B) in zip(mods, ref):
        _check(m["n_out"], W0, A, B, 1.5, f"r{A.shape[0]}")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_module_that_is_not_finite_leaves_the_others_alone(bad):
    mods, ref = [], []
    for i in range(24):
        r = (64, 48, 96, 16)[i % 4]
        W0, A, B = _module(700, 512, r, i)
        if i % 2 == 0:  # the even ones, with wider products, are not finite
            W0[:] = bad
            A[::3] = bad
        ref.append((W0, A, B))
        mods.append(dict(W0=W0.cuda(), A=A.cuda(), B=B.cuda(), s=1.5,
                         n_out=torch.empty(700, device="cuda")))
    dora.dora_factored_norm_grouped(mods)
    for i in range(1, 24, 2):
        _check(mods[i]["n_out"], *ref[i], 1.5, f"module {i}")


@pytest.mark.parametrize("r", [8, 24, 48, 72, 200, 384, 392, 512])
def test_merge_behind_the_int8_product(poison, r):
    W0, A, B = _module(300, 264, r, r)
    m, n = torch.rand(300) + 0.5, torch.rand(300) + 0.5
    Wc, Ac, Bc, mc, nc = (t.cuda() for t in (W0, A, B, m, n))
    poison()
    W = dora.dora_merge_weight(Wc, Ac, Bc, mc, nc, 2.0, 2.0 ** -7)
    ref = oracle.merge_weight_given_norm(_np(W0), _np(A), _np(B), _np(m), _np(n), 2.0, 2.0 ** -7)
    # the bf16 rounding, and fp32 sums of r products (two roundings each)
    g = (_np(m) / np.maximum(_np(n), 2.0 ** -7))[:, None]
    terms = g * (np.abs(_np(W0)) + 2.0 * np.abs(_np(B)) @ np.abs(_np(A)))
    tol = 2.0 ** -8 * np.abs(ref) * 1.01 + (2 * r + 8) * 2.0 ** -24 * terms
    assert (np.abs(_np(W) - ref) <= tol).all()
