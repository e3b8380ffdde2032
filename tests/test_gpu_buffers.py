"""Graphs captured at several sizes of one layer object, replayed after eager
calls at others: the replays give the eager results and touch nobody's memory."""
import pytest
import torch

import synth
from helpers import dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

D, H, E, K = 256, 128, 16, 4
n = lambda shape, i, sc: synth.normal(shape, 17, i, sc)


def _capture(run):
    """run() warmed up on a side stream and captured; the graph and its outputs."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    return graph, out


def _fill(seed):
    """Tensors that take whatever memory was given back, and a check that they stay."""
    ts = [torch.full((1 << k,), seed, dtype=torch.uint8, device="cuda") for k in range(9, 27)]
    ts += [torch.full((1 << 14,), seed, dtype=torch.uint8, device="cuda") for _ in range(200)]
    return ts, lambda: all(bool((t == seed).all()) for t in ts)


def _replays(graphs, inputs, refs, between):
    """Each graph replayed in turn on new inputs against refs(i); eager work between."""
    for i in range(3):
        for (graph, got), x, ref in zip(graphs, inputs, refs):
            x.copy_(dev(n(x.shape, 30 + i, 1.0), x.dtype))
            tensors, untouched = _fill(i + 1)
            graph.replay()
            torch.cuda.synchronize()
            want = ref()
            assert len(want) == len(got)
            for g, w in zip(got, want):
                assert torch.equal(g, w), i
            assert untouched(), i
            del tensors
            between(i)


def test_w4_layer_at_several_sizes(monkeypatch):
    """One graph for each batch size; a prompt of another size between the
    replays. Nothing but what the graphs use is kept here."""
    monkeypatch.setattr(moe, "_KEPT_BYTES", 0)
    w1, w2 = (dev(n(s, 2, 0.05), torch.float32) for s in ((E, 2 * H, D), (E, D, H)))
    layer, eager = moe.MoELayerW4(w1, w2, K), moe.MoELayerW4(w1, w2, K)
    wr = dev(n((E, D), 4, 0.2), torch.float32)
    step = lambda lay, x: (lay.forward(x, x.float() @ wr.t()),)
    inputs = [dev(n((T, D), 5, 1.0), torch.bfloat16) for T in (1, 4)]
    graphs = [_capture(lambda: step(layer, x)) for x in inputs]
    prompt = dev(n((64, D), 6, 1.0), torch.bfloat16)
    step(layer, prompt)
    _replays(graphs, inputs, [lambda x=x: step(eager, x) for x in inputs],
             lambda i: step(layer, prompt[:64 - i]))


@pytest.mark.parametrize("act8", [False, True])
def test_norm_at_several_sizes(monkeypatch, act8):
    monkeypatch.setattr(moe, "_KEPT_BYTES", 0)
    w, b = dev(1 + n((D,), 7, 0.1), torch.float32), dev(n((D,), 8, 0.1), torch.float32)
    norm, eager = (moe.LayerNorm(w, b, act8=act8) for _ in range(2))

    def step(obj, x):
        y = obj.forward(x)
        g = obj.backward(x)
        return y, g["dx"], g["dweight"], g["dbias"]

    inputs = [dev(n((T, D), 5, 1.0), torch.bfloat16) for T in (3, 40)]
    graphs = [_capture(lambda: step(norm, x)) for x in inputs]
    other = dev(n((64, D), 6, 1.0), torch.bfloat16)
    step(norm, other)
    _replays(graphs, inputs, [lambda x=x: step(eager, x) for x in inputs],
             lambda i: step(norm, other[:64 - i]))


def test_w4_weights_change_between_replays():
    """A captured step takes the weights that the layer was given last."""
    w = [[dev(n(s, 2 + i, 0.05), torch.float32) for s in ((E, 2 * H, D), (E, D, H))] for i in range(3)]
    layer = moe.MoELayerW4(*w[0], K)
    x, lg = dev(n((4, D), 5, 1.0), torch.bfloat16), dev(n((4, E), 6, 1.0), torch.float32)
    graph, got = _capture(lambda: layer.forward(x, lg))
    seen = []
    for i in (0, 1, 2, 0):
        layer.prepare_weights(*w[i])
        tensors, untouched = _fill(i + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, moe.MoELayerW4(*w[i], K).forward(x, lg)), i
        assert untouched(), i
        del tensors
        seen.append(got.clone())
    assert torch.equal(seen[0], seen[3]) and not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("kind", ["bf16", "bf16 act8", "bf16 recompute", "mxfp8", "mxfp8 act8", "padded"])
def test_layers_at_several_sizes(monkeypatch, kind):
    """Forward and backward of the layers, with the balancing loss, one graph
    for each micro-batch size."""
    monkeypatch.setattr(moe, "_KEPT_BYTES", 0)
    mx = kind.startswith("mxfp8")
    w1, w2 = (dev(n(s, 2, 0.05), torch.float32 if mx else torch.bfloat16)
              for s in ((E, 2 * H, D), (E, D, H)))
    opt = {kind.split()[1]: True} if " " in kind else {}

    def make():
        if kind == "padded":
            return moe.MoELayerPadded(w1, w2, K, 48)
        norm = moe.LayerNorm(torch.ones(D, device="cuda"), None)
        return (moe.MoELayerMX if mx else moe.MoELayer)(w1, w2, K, aux_alpha=0.01, scratch={},
                                                        out_norm=norm, **opt)

    layer, eager = make(), make()
    wr = dev(n((E, D), 4, 0.2), torch.float32)

    def step(lay, x):
        out = lay.forward(x, x.float() @ wr.t())
        g = lay.backward(x)
        return (out, *(v for v in g.values() if v is not None and v.dtype == torch.float32), g["dx"])

    inputs = [dev(n((T, D), 5, 1.0), torch.bfloat16) for T in (40, 96)]
    graphs = [_capture(lambda: step(layer, x)) for x in inputs]
    other = dev(n((256, D), 6, 1.0), torch.bfloat16)
    step(layer, other)
    _replays(graphs, inputs, [lambda x=x: step(eager, x) for x in inputs],
             lambda i: step(layer, other[:256 - i]))


def test_mxfp8_weights_change_between_replays():
    """A captured training step takes the weights that were quantised last."""
    w = [[dev(n(s, 2 + i, 0.05), torch.float32) for s in ((E, 2 * H, D), (E, D, H))] for i in range(2)]
    layer = moe.MoELayerMX(*w[0], K, scratch={})
    x, lg = dev(n((70, D), 5, 1.0), torch.bfloat16), dev(n((70, E), 6, 1.0), torch.float32)
    names = ("dx", "dw1", "dw2", "dlogits")

    def step(lay):
        out = lay.forward(x, lg)
        g = lay.backward(x)
        return [out, *(g[k] for k in names)]

    graph, got = _capture(lambda: step(layer))
    for i in (1, 0, 1):
        layer.prepare_weights(*w[i])
        tensors, untouched = _fill(i + 1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(moe.MoELayerMX(*w[i], K, scratch={}))):
            assert torch.equal(a, b), i
        assert untouched(), i
        del tensors
