"""The operators as they are used together: a residual stream, the norm with
its 8-bit checkpoint, the router, the checkpointing layer with a norm behind
it, forward and backward; eagerly, captured into a graph, and on streams side
by side."""
import numpy as np
import pytest
import torch

import synth
from helpers import dev, rel_fro, to_np

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

T, D, E, K, HID = 192, 256, 8, 2, 128
EPS = 1e-5


def _data(dt, seed=71):
    n = lambda shape, i, s: synth.normal(shape, seed, i, s)
    return dict(x=dev(n((T, D), 1, 1.0), dt), res=dev(n((T, D), 5, 1.0), dt),
                w1=dev(n((E, 2 * HID, D), 2, 0.08), dt), w2=dev(n((E, D, HID), 3, 0.08), dt),
                dout=dev(n((T, D), 4, 1.0), dt), wr=dev(n((E, D), 6, 0.1), torch.float32),
                g1=dev(1 + n((D,), 7, 0.1), torch.float32), b1=dev(n((D,), 8, 0.1), torch.float32),
                g2=dev(1 + n((D,), 9, 0.1), torch.float32))


class Sublayer:
    """out = s + norm2(experts(norm1(s))), s = x + res; the router reads norm1's output."""

    def __init__(self, v, act8):
        self.v = v
        self.scratch = {}
        self.norm = moe.LayerNorm(v["g1"], v["b1"], EPS, act8=act8)
        self.layer = moe.MoELayer(v["w1"], v["w2"], K, act8=act8, scratch=self.scratch,
                                  out_norm=moe.LayerNorm(v["g2"], None, EPS, act8=act8))

    def forward(self):
        v = self.v
        self.y = self.norm.forward(v["x"], v["res"])
        out = self.layer.forward(self.y, self.y.float() @ v["wr"].t())
        return (self.norm.sum.float() + out.float()).to(out.dtype)

    def backward(self):
        v = self.v
        g = self.layer.backward(v["dout"])
        dy = (g["dx"].float() + g["dlogits"] @ v["wr"]).to(g["dx"].dtype)
        n = self.norm.backward(dy, v["dout"])
        return dict(dx=n["dx"], dg1=n["dweight"], db1=n["dbias"], dw1=g["dw1"], dw2=g["dw2"],
                    dg2=g["dnorm_weight"], dwr=g["dlogits"].t() @ self.y.float())


def _autograd(v, idx):
    """The same in float64 on the CPU, the selection given."""
    p = {k: t.detach().double().cpu().requires_grad_(k not in ("dout",)) for k, t in v.items()}
    s = p["x"] + p["res"]

    def norm(z, w, b):
        m = z - z.mean(1, keepdim=True)
        y = m / torch.sqrt((m * m).mean(1, keepdim=True) + EPS) * w
        return y if b is None else y + b

    y = norm(s, p["g1"], p["b1"])
    gate = torch.softmax(torch.gather(y @ p["wr"].t(), 1, idx), 1)
    rows = []
    for j in range(K):
        w1, w2 = p["w1"][idx[:, j]], p["w2"][idx[:, j]]
        ab = torch.einsum("td,tnd->tn", y, w1)
        h = torch.nn.functional.silu(ab[:, :HID]) * ab[:, HID:]
        rows.append(gate[:, j:j + 1] * torch.einsum("th,tdh->td", h, w2))
    out = s + norm(sum(rows), p["g2"], None)
    out.backward(p["dout"])
    return out.detach(), dict(dx=p["x"].grad, dg1=p["g1"].grad, db1=p["b1"].grad, dw1=p["w1"].grad,
                              dw2=p["w2"].grad, dg2=p["g2"].grad, dwr=p["wr"].grad)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act8", [False, True])
def test_against_autograd(dt, act8):
    """Whole-tensor Frobenius errors. fp32 without checkpoints: sums of at
    most 256 products and a few norms, 1e-5. A checkpoint's element is off by
    a step / sqrt(12), the step at most amax (about 2.1 deviations of 32
    normals) / 64: 1 %; a gradient meets five checkpointed factors (the norms'
    xh, a, b, y, dH'), in quadrature under 3 %. bf16's roundings (2^-8 at most)
    along a dozen stored tensors: 1 %; a token whose selection bf16 changes
    would break this, so the float64 run is given the layer's."""
    v = _data(dt)
    sub = Sublayer(v, act8)
    out = sub.forward()
    g = sub.backward()
    idx = sub.layer.route["topk_idx"].long().cpu()
    ref, rg = _autograd(v, idx)
    base = 1e-5 if dt == torch.float32 else 0.01
    assert rel_fro(to_np(out), ref.numpy()) <= base
    for k, t in rg.items():
        assert rel_fro(to_np(g[k]), t.numpy()) <= base + (0.03 if act8 else 0.0), k


def _run(sub):
    out = sub.forward()
    return dict(sub.backward(), out=out)


def test_graph_replays():
    """Forward and backward captured once and replayed on new inputs, with
    eager runs of another sublayer and synchronisations between the replays."""
    v = _data(torch.bfloat16)
    sub, eager = Sublayer(v, True), Sublayer(v, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            _run(sub)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(sub)
    for i in range(4):
        v["x"].copy_(dev(synth.normal((T, D), 80 + i, 1, 1.0), torch.bfloat16))
        v["dout"].copy_(dev(synth.normal((T, D), 80 + i, 4, 1.0), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        ref = {k: t.clone() for k, t in _run(eager).items()}
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(got[k], ref[k]), (i, k)


def test_streams_side_by_side():
    """Two sublayers with scratch of their own, on two streams at once, give
    what each gives alone; calls follow the current stream."""
    vs = [_data(torch.bfloat16, s) for s in (91, 92)]
    alone = [{k: t.clone() for k, t in _run(Sublayer(v, True)).items()} for v in vs]
    subs = [Sublayer(v, True) for v in vs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _run(subs[i])
    torch.cuda.synchronize()
    for i in range(2):
        for k in alone[i]:
            assert torch.equal(got[i][k], alone[i][k]), (i, k)


def test_same_bits_every_time():
    v = _data(torch.bfloat16)
    sub = Sublayer(v, True)
    first = {k: t.clone() for k, t in _run(sub).items()}
    for _ in range(3):
        again = _run(sub)
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_one_token_without_a_backward():
    """The norm's serving form in front of one token's layer."""
    v = _data(torch.bfloat16)
    x, r = v["x"][:1].contiguous(), v["res"][:1].contiguous()
    whole = moe.moe_layer_norm(v["x"], v["g1"], v["b1"], EPS, residual=v["res"])
    one = moe.moe_layer_norm(x, v["g1"], v["b1"], EPS, residual=r, stats=False)
    assert torch.equal(one["y"], whole["y"][:1]) and torch.equal(one["sum"], whole["sum"][:1])


@pytest.mark.parametrize("kind", ["bf16", "bf16 act8", "mxfp8 act8"])
def test_micro_batches_accumulate(kind):
    """Two backward passes of one forward, the second added to the first: the
    weight gradients, the norm's among them, are exactly doubled (the same
    sum twice, one fp32 addition), dx and the rest as before."""
    v = _data(torch.bfloat16)
    act8 = kind.endswith("act8")
    norm = moe.LayerNorm(v["g2"], v["b1"], EPS, act8=act8)
    make = moe.MoELayerMX if kind.startswith("mxfp8") else moe.MoELayer
    w = (v["w1"].float(), v["w2"].float()) if make is moe.MoELayerMX else (v["w1"], v["w2"])
    layer = make(*w, K, act8=act8, scratch={}, out_norm=norm)
    layer.forward(v["x"], v["x"].float() @ v["wr"].t())
    with pytest.raises(ValueError, match="earlier backward"):
        layer.backward(v["dout"], accumulate_dw=True)
    names = ("dx", "dlogits", "dw1", "dw2", "dnorm_weight", "dnorm_bias")
    g = layer.backward(v["dout"])
    one = {n: g[n].clone() for n in names}
    g = layer.backward(v["dout"], accumulate_dw=True)
    for n in names:
        assert torch.equal(g[n], one[n] * (2 if n.startswith(("dw", "dnorm")) else 1)), n
    g = layer.backward(v["dout"])
    for n in names:
        assert torch.equal(g[n], one[n]), n
