"""A product right behind the kernels that write its operands, on the same
buffers with new contents each time: its early prefetch of the weight and its
launch ahead of their end must not show.  Eager and captured; bit for bit with
calls that are waited for one by one."""
import pytest
import torch

import dora_adapter_factored_b200 as dora

pytestmark = pytest.mark.gpu


def _rand(rows, cols, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, cols, device="cuda", generator=g) * scale).bfloat16()


@pytest.mark.parametrize("T,d_out,d_in", [(1, 4096, 4096), (24, 8192, 8192), (64, 1024, 8192),
                                          (333, 2048, 4096), (1500, 2048, 2048), (9, 1001, 1003)])
def test_weights_and_tokens_written_right_before(T, d_out, d_in):
    W = [_rand(d_out, d_in, s, 0.02) for s in range(3)]
    x = [_rand(T, d_in, 10 + s) for s in range(3)]
    gain = _rand(1, d_in, 20)[0].contiguous()
    want = []
    for s in range(3):
        wq, sw = dora.dora_quantize_rows(W[s])
        xq, sx, _ = dora.dora_rmsnorm_quant(x[s], gain, 1e-6, residual=x[s])
        torch.cuda.synchronize()
        want.append(dora.dora_linear_i8(xq, sx, wq, sw))
        torch.cuda.synchronize()
    wq = torch.zeros(d_out, d_in, dtype=torch.int8, device="cuda")
    sw, sx = torch.zeros(d_out, device="cuda"), torch.zeros(T, device="cuda")
    xq = torch.zeros(T, d_in, dtype=torch.int8, device="cuda")
    h = torch.empty(T, d_in, dtype=torch.bfloat16, device="cuda")
    y = [torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda") for _ in range(30)]

    def run():
        for i in range(30):
            s = i % 3
            # the weight's writer directly before the product, and the tokens' in turn
            if i % 2:
                dora.dora_rmsnorm_quant(x[s], gain, 1e-6, residual=x[s], h_out=h, q=xq, scale=sx)
                dora.dora_quantize_rows(W[s], q=wq, scale=sw)
            else:
                dora.dora_quantize_rows(W[s], q=wq, scale=sw)
                dora.dora_rmsnorm_quant(x[s], gain, 1e-6, residual=x[s], h_out=h, q=xq, scale=sx)
            dora.dora_linear_i8(xq, sx, wq, sw, y=y[i])

    run()
    torch.cuda.synchronize()
    assert all(torch.equal(y[i], want[i % 3]) for i in range(30))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in y:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y[i], want[i % 3]) for i in range(30))
    assert dora.dora_get_device_status() == 0


def test_norm_merge_and_products_in_turn():
    """The whole path again and again without a wait in between: each call leaves
    shared and tensor memory to the next."""
    shapes = [(512, 256, 16), (1024, 512, 48), (300, 768, 384), (2048, 1024, 72)]
    mods = []
    for k, (d_out, d_in, r) in enumerate(shapes):
        A, B = _rand(r, d_in, k, d_in ** -0.5), _rand(d_out, r, k + 5, 0.02)
        mods.append((_rand(d_out, d_in, k + 9, 0.02), A, B, torch.rand(d_out, device="cuda") + 0.5))
    x = {d_in: _rand(700, d_in, d_in) for _, d_in, _ in shapes}

    def chain(W0, A, B, m, T):
        n, g = dora.dora_factored_norm(W0, A, B, 2.0, m, 2.0 ** -7)
        W = dora.dora_merge_weight(W0, A, B, m, n, 2.0, 2.0 ** -7)
        wq, sw = dora.dora_quantize_rows(W)
        xq, sx = dora.dora_quantize_rows(x[W0.shape[1]][:T])
        y = dora.dora_linear_i8(xq, sx, wq, sw, dtype=torch.float32)
        n2, _ = dora.dora_factored_norm(dora.dora_dequantize_rows(wq, sw), A, B, 2.0)
        return n, g, W, wq, sw, y, n2

    want = []
    for T in (3, 60, 700):
        for mod in mods:
            want.append([t.clone() for t in chain(*mod, T)])
            torch.cuda.synchronize()
    for _ in range(4):
        got = [chain(*mod, T) for T in (3, 60, 700) for mod in mods]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert dora.dora_get_device_status() == 0
