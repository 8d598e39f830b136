"""Measured cases of the 8-bit serving operators of a merged DoRA weight.

Three operators: the quantisation of a matrix by rows (a merged weight's
output channels, or activations per token), the RMS norm with the residual's
addition and 8-bit output, and the linear layer on 8-bit operands with a scale
per token and per output channel.  `own` false runs them in plain torch
operations, true through the library.  8-bit results are returned as the
values they stand for (code times scale, in bf16), next to the fp32 scales.
"""
import math

import torch

own = False

EPS = 1e-6
MAX_NORM_ELEMS = 8192 * 8192       # largest listed norm
MAX_QUANT_ELEMS = 25600 * 5120     # largest listed quantisation
MAX_LINEAR_MACS = 4096 * 8192 * 8192  # largest listed linear layer

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token between two layers of a decoding step: pure latency.
        dict(name="norm_1x4096", op="norm", T=1, d=4096, dt="bf16", residual=True),
        # A decoding batch of odd size at the rectangular workload's width.
        dict(name="norm_203x5120", op="norm", T=203, d=5120, dt="bf16", residual=True),
        # The first norm of an fp32 model, no residual yet; a width no vector divides.
        dict(name="norm_2047x4099_f32", op="norm", T=2047, d=4099, dt="f32", residual=False),
        # A long prefill at the headline width.
        dict(name="norm_8192x8192", op="norm", T=8192, d=8192, dt="bf16", residual=True),
        # Input of a down projection (no norm before it) for a small fp32 batch.
        dict(name="quant_37x14336_f32", op="quant", T=37, d=14336, dt="f32"),
        # A merged k/v projection, quantised when an adapter is loaded.
        dict(name="quant_1024x4096", op="quant", T=1024, d=4096, dt="bf16"),
        # The merged rectangular up projection.
        dict(name="quant_25600x5120", op="quant", T=25600, d=5120, dt="bf16"),
        # One token through an up projection of the layer stack: the weight's stream.
        dict(name="linear_1x14336x4096", op="linear", T=1, d_out=14336, d_in=4096, dt="bf16",
             bias=False),
        # A decoding batch through the headline module.
        dict(name="linear_24x8192x8192", op="linear", T=24, d_out=8192, d_in=8192, dt="bf16",
             bias=False),
        # Ragged everywhere: rows of the operands start at any byte.
        dict(name="linear_77x1001x1003_f32", op="linear", T=77, d_out=1001, d_in=1003, dt="f32",
             bias=True),
        # An odd prompt through a down projection with a bias.
        dict(name="linear_333x4096x14336", op="linear", T=333, d_out=4096, d_in=14336, dt="bf16",
             bias=True),
        # A full prefill through the headline module: the tensor cores' case.
        dict(name="linear_4096x8192x8192", op="linear", T=4096, d_out=8192, d_in=8192, dt="bf16",
             bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A width: three in four a multiple of `step`, the others any number."""
    d = _log_int(rng, lo, hi)
    return max(step, d // step * step) if rng.random() < 0.75 else d


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "linear", "linear", "linear"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        d_in = _width(rng, 64, 14336, 16)
        d_out = _width(rng, 64, 25600, 8)
        T = _log_int(rng, 1, max(1, min(8192, MAX_LINEAR_MACS // (d_in * d_out))))
        return dict(op=op, T=T, d_out=d_out, d_in=d_in, dt=dt, bias=rng.random() < 0.3)
    # fp32 elements cost twice the bytes of the listed bf16 cases
    size = 2 if dt == "f32" else 1
    d = _width(rng, 64, 16384, 8)
    if op == "quant":
        T = _log_int(rng, 1, min(25600, MAX_QUANT_ELEMS // (d * size)))
        return dict(op=op, T=T, d=d, dt=dt)
    T = _log_int(rng, 1, min(8192, MAX_NORM_ELEMS // (d * size)))
    return dict(op=op, T=T, d=d, dt=dt, residual=rng.random() < 0.75)


def _hidden(T, d, g):
    """Hidden states: unit rows with a few strong channels."""
    gain = torch.ones(d, device="cuda")
    strong = torch.rand(d, device="cuda", generator=g) < 0.004
    gain[strong] = 12.0
    return torch.randn(T, d, device="cuda", generator=g) * gain


def _codes(x):
    """int8 codes and scales of the rows of x, as any quantiser gives them."""
    amax = x.abs().amax(dim=1).clamp_min(1e-20)
    return torch.round(x * (127.0 / amax)[:, None]).to(torch.int8), amax / 127.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dt"]]
    T = case["T"]
    if case["op"] == "norm":
        d = case["d"]
        return dict(op="norm", x=_hidden(T, d, g).to(dt),
                    residual=(3.0 * _hidden(T, d, g)).to(dt) if case["residual"] else None,
                    weight=(1.0 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt))
    if case["op"] == "quant":
        return dict(op="quant", x=(0.02 * _hidden(T, case["d"], g)).to(dt))
    d_out, d_in = case["d_out"], case["d_in"]
    xq, sx = _codes(_hidden(T, d_in, g))
    wq, sw = _codes(0.02 * torch.randn(d_out, d_in, device="cuda", generator=g))
    bias = 0.5 * torch.randn(d_out, device="cuda", generator=g) if case["bias"] else None
    return dict(op="linear", xq=xq, sx=sx, wq=wq, sw=sw, bias=bias, dt=dt)


def _run_own(s):
    import dora_adapter_factored_b200 as dora
    if s["op"] == "norm":
        q, scale, h = dora.dora_rmsnorm_quant(s["x"], s["weight"], EPS, residual=s["residual"])
        return dict(values=dora.dora_dequantize_rows(q, scale), scale=scale, h=h)
    if s["op"] == "quant":
        q, scale = dora.dora_quantize_rows(s["x"])
        return dict(values=dora.dora_dequantize_rows(q, scale), scale=scale)
    return dict(y=dora.dora_linear_i8(s["xq"], s["sx"], s["wq"], s["sw"], bias=s["bias"],
                                      dtype=s["dt"]))


def _plain_rows(v):
    """Codes (in fp32) and scales of the rows of v."""
    amax = v.abs().amax(dim=1)
    return torch.round(v * (127.0 / amax)[:, None]), amax / 127.0


def _run_plain(s):
    if s["op"] == "norm":
        x, h = s["x"].float(), None
        if s["residual"] is not None:
            h = (x + s["residual"].float()).to(s["x"].dtype)
            x = h.float()
        v = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        q, scale = _plain_rows(v)
        return dict(values=(q * scale[:, None]).bfloat16(), scale=scale, h=h)
    if s["op"] == "quant":
        q, scale = _plain_rows(s["x"].float())
        return dict(values=(q * scale[:, None]).bfloat16(), scale=scale)
    y = (s["xq"].float() @ s["wq"].float().t()) * s["sx"][:, None] * s["sw"][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return dict(y=y.to(s["dt"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    es = 2 if case["dt"] == "bf16" else 4
    T = case["T"]
    if case["op"] == "linear":
        d_out, d_in = case["d_out"], case["d_in"]
        nbytes = T * d_in + d_out * d_in + 4 * T + 4 * d_out + T * d_out * es
        return {"bytes": nbytes + (4 * d_out if case["bias"] else 0),
                "flops": 2 * T * d_out * d_in}
    d = case["d"]
    if case["op"] == "quant":
        return {"bytes": T * d * (es + 1) + 4 * T, "flops": 3 * T * d}
    streams = 3 if case["residual"] else 1
    return {"bytes": T * d * (streams * es + 1) + d * es + 4 * T, "flops": 7 * T * d}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        # integer sums below 2^53 are exact in 64-bit floating point
        out = torch.matmul(s["xq"].double(), s["wq"].double().transpose(0, 1))
        out *= torch.outer(s["sx"].double(), s["sw"].double())
        if s["bias"] is not None:
            out += s["bias"].double()[None, :]
        return dict(y=out)
    h = None
    if s["op"] == "norm":
        u = s["x"].double()
        if s["residual"] is not None:
            h = u + s["residual"].double()
            u = h.to(s["x"].dtype).double()  # the norm is of the stored sum
        rms = torch.sqrt(u.square().sum(dim=1) / u.shape[1] + EPS)
        u = u / rms[:, None] * s["weight"].double()[None, :]
    else:
        u = s["x"].double()
    top = torch.linalg.vector_norm(u, ord=math.inf, dim=1)
    step = top / 127
    values = torch.round(u / step[:, None]) * step[:, None]
    if s["op"] == "norm":
        return dict(values=values, scale=step, h=h)
    return dict(values=values, scale=step)
