"""CPU-side checks of the 8-bit serving calls: the oracle's own pins, host
validation before any launch, and what the binding refuses."""
import ctypes

import numpy as np
import pytest
import torch

import dora_adapter_factored_b200 as dora
import oracle
from dora_adapter_factored_b200 import _abi

vp = ctypes.c_void_p
X, R, W, H, Q, S = (vp(0x1000000 * (i + 1)) for i in range(6))
F32, BF16 = _abi.DORA_F32, _abi.DORA_BF16
INVALID, UNSUPPORTED = _abi.DORA_ERR_INVALID_ARG, _abi.DORA_ERR_UNSUPPORTED


# ------------------------------------------------------------------ oracle

def test_oracle_codes_by_hand():
    q, scale, _ = oracle.quantize_rows([[127.0, -127.0, 0.5, 1.5, -2.5, 0.49],
                                        [0.0, 0.0, 0.0, 0.0, 0.0, 0.0],
                                        [1.0, np.inf, 0.0, 0.0, 0.0, 0.0],
                                        [1.0, np.nan, 0.0, 0.0, 0.0, 0.0]])
    assert q[0].tolist() == [127, -127, 0, 2, -2, 0]  # halves to even
    assert scale[0] == 1.0 and scale[1] == 0.0
    assert np.isnan(scale[2]) and np.isnan(scale[3])
    assert not q[1:].any()


def test_oracle_norm_and_linear_by_hand():
    v = oracle.rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0)
    assert np.allclose(v, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    acc, y = oracle.linear_i8([[1, -2], [3, 4]], [0.5, 2.0], [[5, 6], [-7, 8], [0, 1]],
                              [1.0, 10.0, 100.0], [0.0, 1.0, 2.0])
    assert acc.tolist() == [[-7, -23, -2], [39, 11, 4]]
    assert y.tolist() == [[-3.5, -114.0, -98.0], [78.0, 221.0, 802.0]]


# -------------------------------------------------------------- validation

def _quant(lib, x=X, dt=BF16, rows=4, cols=64, q=Q, scale=S):
    return lib.dora_quantize_rows(x, dt, rows, cols, q, scale, None)


def _deq(lib, q=Q, scale=S, dt=BF16, rows=4, cols=64, x=X):
    return lib.dora_dequantize_rows(q, scale, dt, rows, cols, x, None)


def _norm(lib, x=X, r=R, w=W, eps=1e-6, dt=BF16, T=4, d=64, h=H, q=Q, scale=S):
    return lib.dora_rmsnorm_quant(x, r, w, eps, dt, T, d, h, q, scale, None)


def _linear(lib, xq=X, sx=R, wq=W, sw=S, bias=None, dt=BF16, T=4, d_out=64, d_in=64, y=H,
            ws=vp(0x9000000), nws=1 << 30):
    return lib.dora_linear_i8(xq, sx, wq, sw, bias, dt, T, d_out, d_in, y, ws, nws, None)


BAD_QUANT = [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(dt=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=(1 << 30) + 1), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(x=vp(0x1000001)), INVALID),             # bf16 at an odd address
    (dict(x=vp(0x1000002), dt=F32), INVALID),     # fp32 at a 2-byte address
    (dict(scale=vp(0x6000002)), INVALID),
    (dict(q=vp(0x1000000)), INVALID),             # codes over x
    (dict(q=vp(0x10001ff)), INVALID),             # ... over its last byte
    (dict(scale=vp(0x1000004)), INVALID),         # scale over x
    (dict(scale=vp(0x5000004)), INVALID),         # scale over the codes
]
BAD_DEQ = [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(dt=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=(1 << 30) + 1), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(x=vp(0x1000001)), INVALID), (dict(x=vp(0x1000002), dt=F32), INVALID),
    (dict(scale=vp(0x6000002)), INVALID), (dict(x=Q), INVALID), (dict(x=S), INVALID),
]
BAD_NORM = [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(q=None), INVALID),
    (dict(scale=None), INVALID), (dict(dt=-1), INVALID), (dict(T=-1), INVALID),
    (dict(d=0), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(r=None), INVALID), (dict(h=None), INVALID),  # a residual without h, and h alone
    (dict(d=(1 << 30) + 1), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
    (dict(h=vp(0x1000010)), INVALID), (dict(h=vp(0x2000010)), INVALID),  # shifted over x, residual
    (dict(h=W), INVALID), (dict(q=X), INVALID), (dict(q=R), INVALID), (dict(q=W), INVALID),
    (dict(q=H), INVALID), (dict(scale=X), INVALID), (dict(scale=H), INVALID),
    (dict(scale=Q), INVALID), (dict(scale=W), INVALID),
]
BAD_LINEAR = [
    (dict(xq=None), INVALID), (dict(sx=None), INVALID), (dict(wq=None), INVALID),
    (dict(sw=None), INVALID), (dict(y=None), INVALID), (dict(dt=3), INVALID),
    (dict(T=-1), INVALID), (dict(d_out=0), INVALID), (dict(d_in=0), INVALID),
    (dict(d_in=131072), UNSUPPORTED),               # the int32 sum could overflow
    (dict(T=(1 << 23) + 1), UNSUPPORTED), (dict(d_out=(1 << 30) + 1), UNSUPPORTED),
    (dict(y=X), INVALID), (dict(y=W), INVALID), (dict(y=R), INVALID), (dict(y=S), INVALID),
    (dict(bias=H), INVALID), (dict(bias=vp(0x7000001)), INVALID), (dict(sx=vp(0x2000002)), INVALID),
    (dict(y=vp(0x4000001)), INVALID), (dict(y=vp(0x4000002), dt=F32), INVALID),
]


@pytest.mark.parametrize("call,bad", [(_quant, BAD_QUANT), (_deq, BAD_DEQ), (_norm, BAD_NORM),
                                      (_linear, BAD_LINEAR)],
                         ids=["quantize", "dequantize", "norm", "linear"])
def test_host_validation(built_library, call, bad):
    lib = dora.load_library(built_library)
    before = dora.dora_launch_count()
    for kw, want in bad:
        assert call(lib, **kw) == want, kw
    assert dora.dora_launch_count() == before


def test_linear_workspace(built_library):
    """Copies with rows of 128-byte steps, where the tensor-core path needs them."""
    lib = dora.load_library(built_library)
    size = dora.dora_linear_i8_workspace_size
    assert size(1, 1000, 1003) == 0 and size(300, 1000, 1008) == 0
    assert size(8, 69, 300) == 0 and size(1, 14336, 4097) > 0 and size(1, 8, 5001) > 0
    need = size(300, 1000, 1003)
    assert need == 300 * 1024 + 1000 * 1024
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (9, 8, 131072)):
        assert size(*bad) == 0
    kw = dict(T=300, d_out=1000, d_in=1003)
    ws = vp(0x9000000)
    for bad in (dict(ws=None), dict(nws=need - 1), dict(ws=vp(0x9000010))):
        assert _linear(lib, **kw, **bad) == _abi.DORA_ERR_WORKSPACE, bad
    for over in (X, R, W, S, H):
        assert _linear(lib, **kw, ws=over) == INVALID
    assert _linear(lib, **kw, bias=ws) == INVALID


def test_valid_arguments_reach_the_device_check(built_library):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = dora.load_library(built_library)
    for call, kws in ((_quant, [{}, dict(rows=0, x=None, q=None, scale=None)]),
                      (_deq, [{}, dict(rows=0, x=None, q=None, scale=None)]),
                      (_norm, [{}, dict(h=X), dict(h=R), dict(r=None, h=None),
                               dict(T=0, x=None, r=None, h=None, q=None, scale=None)]),
                      (_linear, [{}, dict(bias=vp(0x7000000)), dict(d_in=131071),
                                 dict(T=0, xq=None, sx=None, y=None)])):
        for kw in kws:
            assert call(lib, **kw) == _abi.DORA_ERR_CUDA, kw


# ----------------------------------------------------------------- binding

def test_binding_refusals(built_library):
    dora.load_library(built_library)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dora.dora_quantize_rows(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dora.dora_rmsnorm_quant(x, x[0], 1e-6)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dora.dora_linear_i8(x.char(), torch.ones(4), x.char(), torch.ones(4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dora.dora_dequantize_rows(x.char(), torch.ones(4))
    with pytest.raises(TypeError, match="torch.Tensor"):
        dora.dora_quantize_rows([[1.0]])
