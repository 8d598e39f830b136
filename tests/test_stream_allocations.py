"""What a call allocates belongs to the stream it runs on.  A workspace that the
call drops on its return would otherwise be handed to the next call of another
stream while its kernels still write it."""
import random

import pytest
import torch

import dora_adapter_factored_b200 as dora

pytestmark = pytest.mark.gpu


def _calls():
    g = torch.Generator().manual_seed(4)
    bf = lambda *n: (0.1 * torch.randn(*n, generator=g)).bfloat16().cuda()
    W0, A, B = bf(300, 256), bf(16, 256), bf(300, 16)
    m, n = torch.rand(300).cuda() + 0.5, torch.rand(300).cuda() + 0.5
    base, lora, dy = bf(40, 300), bf(40, 300), bf(40, 300)
    k = (m, n, 2.0, 0.01)
    grouped = [dict(W0=W0, A=A, B=B, s=2.0, n_out=torch.empty(300, device="cuda"))]
    comp = [dict(dy=dy, base=base, lora=lora, m=m, n=n, s=2.0, d_base=torch.empty_like(dy),
                 d_lora=torch.empty_like(dy), dm=torch.empty(300, device="cuda"))]
    xq, sx = dora.dora_quantize_rows(base)
    odd = xq[:, :299].contiguous()
    w = base[0].contiguous()
    return {
        "norm": lambda st: dora.dora_factored_norm(W0, A, B, 2.0, m, 0.01, stream=st),
        "norm, grouped": lambda st: dora.dora_factored_norm_grouped(grouped, stream=st),
        "norm, squared": lambda st: dora.dora_factored_norm_sq(W0, A, B, 2.0, stream=st),
        "finalize": lambda st: dora.dora_norm_finalize(n, m, 0.01, stream=st),
        "forward": lambda st: dora.dora_compose_fwd(base, lora, *k, stream=st),
        "delta": lambda st: dora.dora_compose_fwd_delta(base, lora, *k, stream=st),
        "training forward": lambda st: dora.dora_compose_fwd_train(base, lora, *k, stream=st),
        "backward": lambda st: dora.dora_compose_bwd(dy, base, lora, *k, stream=st),
        "static backward": lambda st: dora.dora_compose_bwd_static(dy, base, lora, *k, stream=st),
        "backward from inner": lambda st: dora.dora_compose_bwd_inner(dy, base, *k, stream=st),
        "frozen backward": lambda st: dora.dora_compose_bwd_frozen(dy, *k, stream=st),
        "backward, grouped": lambda st: dora.dora_compose_bwd_grouped(comp, stream=st),
        "merge": lambda st: dora.dora_merge_weight(W0, A, B, *k, stream=st),
        "quantise": lambda st: dora.dora_quantize_rows(base, stream=st),
        "dequantise": lambda st: dora.dora_dequantize_rows(xq, sx, stream=st),
        "norm, quantised": lambda st: dora.dora_rmsnorm_quant(base, w, 1e-6, residual=base,
                                                              stream=st),
        "linear": lambda st: dora.dora_linear_i8(odd, sx, odd, sx, stream=st),
    }


@pytest.mark.parametrize("how", ["Stream", "handle"])
def test_every_allocation_is_the_streams(monkeypatch, how):
    side = torch.cuda.Stream()
    calls = _calls()
    torch.cuda.synchronize()
    seen = []

    def watched(make):
        def call(*a, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return make(*a, **kw)
        return call
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    for name, call in calls.items():
        seen.clear()
        call(side if how == "Stream" else side.cuda_stream)
        torch.cuda.synchronize()
        assert set(seen) <= {side.cuda_stream}, name
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        seen.clear()
        call(None)
        assert set(seen) <= {torch.cuda.default_stream().cuda_stream}, name
    torch.cuda.synchronize()


def test_calls_on_many_streams_at_once():
    """Norms, merges, backward passes and products that overlap on five streams,
    each with the workspace that the binding gave it: the bits of calls alone."""
    g = torch.Generator("cuda").manual_seed(1)
    bf = lambda s, *n: (s * torch.randn(*n, device="cuda", generator=g)).bfloat16()
    jobs = []
    for d_out, d_in, r in ((2048, 1024, 48), (1024, 4096, 384), (513, 1000, 96)):
        W0, A, B = bf(0.02, d_out, d_in), bf(0.03, r, d_in), bf(0.02, d_out, r)
        m = torch.rand(d_out, device="cuda", generator=g) + 0.5
        jobs.append(lambda st, a=(W0, A, B, 2.0, m, 1e-3): dora.dora_factored_norm(*a, stream=st))
        jobs.append(lambda st, a=(W0, A, B, m, m, 2.0, 1e-3): (dora.dora_merge_weight(*a, stream=st),))
        t = (bf(1.0, 700, d_out), bf(1.0, 700, d_out), bf(1.0, 700, d_out), m, m, 2.0, 1e-3)
        jobs.append(lambda st, t=t: dora.dora_compose_bwd(*t, stream=st))
    for T, d_out, d_in in ((24, 8192, 1024), (77, 1001, 1003), (333, 2048, 4096)):
        codes = lambda r, c: torch.randint(-128, 128, (r, c), dtype=torch.int8, device="cuda",
                                           generator=g)
        a = (codes(T, d_in), torch.rand(T, device="cuda", generator=g), codes(d_out, d_in),
             torch.rand(d_out, device="cuda", generator=g))
        jobs.append(lambda st, a=a: (dora.dora_linear_i8(*a, stream=st),))
    want = [[t.clone() for t in job(None)] for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    rng = random.Random(3)
    wrong = 0
    for _ in range(40):
        out = []
        for _ in range(50):
            i = rng.randrange(len(jobs))
            out.append((i, jobs[i](rng.choice(streams))))
        torch.cuda.synchronize()
        wrong += sum(not all(torch.equal(a, b) for a, b in zip(o, want[i])) for i, o in out)
        assert dora.dora_get_device_status() == 0
    assert wrong == 0, f"{wrong} of 2000 calls"
