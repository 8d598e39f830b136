"""The grouped norm captured into a graph: its table of modules has to live as
long as the graph, through replays on new inputs, after the host's memory has
been used for other things, and after other grouped calls."""
import gc

import pytest
import torch

import dora_adapter_factored_b200 as dora

pytestmark = pytest.mark.gpu

SHAPES = [(300, 256, 16), (1000, 512, 384), (513, 320, 48), (64, 1024, 8), (2048, 256, 264)]


def _modules(seed, count):
    g = torch.Generator("cuda").manual_seed(seed)
    bf = lambda s, *n: (s * torch.randn(*n, device="cuda", generator=g)).bfloat16()
    out = []
    for i in range(count):
        d_out, d_in, r = SHAPES[i % len(SHAPES)]
        out.append(dict(W0=bf(0.02, d_out, d_in), A=bf(0.03, r, d_in), B=bf(0.02, d_out, r), s=1.5,
                        m=torch.rand(d_out, device="cuda", generator=g) + 0.5,
                        n_out=torch.zeros(d_out, device="cuda"),
                        g_out=torch.zeros(d_out, device="cuda")))
    return out


def _results(mods):
    return [t.clone() for m in mods for t in (m["n_out"], m["g_out"])]


@pytest.mark.parametrize("count", [1, 5, 56])
@pytest.mark.parametrize("own_ws", [True, False])
def test_captured_and_replayed(count, own_ws):
    mods, other = _modules(1, count), _modules(2, count)
    dora.dora_factored_norm_grouped(other, 0.01)
    want_other = _results(other)
    dora.dora_factored_norm_grouped(mods, 0.01)
    want = _results(mods)
    ws = torch.empty(dora.dora_factored_norm_grouped_workspace_size(mods), dtype=torch.uint8,
                     device="cuda") if own_ws else None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dora.dora_factored_norm_grouped(mods, 0.01, ws=ws)
    # the host's freed memory is used for other things
    hold = [bytearray(b"\xff" * n) for n in (4096, 16384, 65536, 131072) for _ in range(20)]
    for _ in range(3):
        for m in mods:
            m["n_out"].zero_()
            m["g_out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_results(mods), want))
        del hold
        gc.collect()
        hold = [bytearray(b"\xff" * n) for n in (1024, 8192, 32768) for _ in range(40)]
        dora.dora_factored_norm_grouped(_modules(3, count), 0.01)
    # new inputs in place
    for m, o in zip(mods, other):
        for k in ("W0", "A", "B", "m"):
            m[k].copy_(o[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(_results(mods), want_other))
    assert dora.dora_get_device_status() == 0


def test_two_graphs_of_different_modules():
    a, b = _modules(5, 7), _modules(6, 12)
    want = []
    for mods in (a, b):
        dora.dora_factored_norm_grouped(mods)
        want.append(_results(mods))
    graphs = []
    for mods in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dora.dora_factored_norm_grouped(mods)
        graphs.append(graph)
    for _ in range(3):
        for mods, graph, ref in zip((a, b), graphs, want):
            for m in mods:
                m["n_out"].zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(m["n_out"], r) for m, r in zip(mods, ref[::2]))
    del graphs[0]
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(m["n_out"], r) for m, r in zip(b, want[1][::2]))
    assert dora.dora_get_device_status() == 0
