"""The gradients' norm and their clipping on the GPU against 64-bit sums.

Tolerances: squares and sums are fp64 (2^-53 a rounding, nothing beside the
rest), the norm is rounded once to fp32: u = 2^-24 relative, 2 u with the fp64
sums. The factor is rounded once to fp32 (u) and the product once to its type
(h, half a step relative to the value, or half of the smallest subnormal)."""
import math

import numpy as np
import pytest
import torch

import synth
from helpers import dev, to_np

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
F32, BF16 = torch.float32, torch.bfloat16


def _norm64(ts):
    return math.sqrt(sum(float((to_np(t).astype(np.float64) ** 2).sum()) for t in ts))


def _check(got, src, norm, max_norm):
    scale = min(1.0, max_norm / (norm + 1e-6))
    for i, (o, g) in enumerate(zip(got, src)):
        want = to_np(g).astype(np.float64) * scale
        tol = np.abs(want) * (H[g.dtype] + 2 * U) + TINY[g.dtype]
        assert (np.abs(to_np(o).astype(np.float64) - want) <= tol).all(), (i, tuple(g.shape), g.dtype)


def _tensors(sizes, dts, seed, pad=0):
    """Tensors one after the other in a flat buffer a type, `pad` elements in
    front of each and behind the last."""
    flats, out = {}, []
    for dt in set(dts):
        n = sum(s + pad for s, t in zip(sizes, dts) if t is dt) + pad
        flats[dt] = dev(synth.normal((max(n, 1),), seed, 0 if dt is F32 else 1, 1.0), dt)
    at = {dt: pad for dt in flats}
    for s, dt in zip(sizes, dts):
        out.append(flats[dt][at[dt]:at[dt] + s])
        at[dt] += s + pad
    return out, flats


# chunks are 8192 fp32 or 16384 bf16 elements, vectors 4 or 8
SIZES = [1, 0, 3, 4, 5, 7, 8, 9, 255, 1023, 4097, 8191, 8192, 8193, 16383, 16384, 16385, 40000, 2, 100001]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("pad", [0, 1, 3])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
def test_sizes_and_places(kind, pad, max_norm):
    """Sizes around the vectors' and the chunks' ends at any element's
    address: the norm alone, in place, into other tensors and with a given
    norm; what lies between the tensors stays."""
    dts = [{"f32": F32, "bf16": BF16}.get(kind) or (F32 if i % 3 else BF16) for i in range(len(SIZES))]
    g, flats = _tensors(SIZES, dts, 5 + pad, pad)
    norm = _norm64(g)
    n = moe.moe_grad_norm(g)
    assert n.shape == () and abs(float(n) - norm) <= 2 * U * norm
    src = [t.clone() for t in g]
    before = {dt: f.clone() for dt, f in flats.items()}
    o, oflats = _tensors(SIZES, dts, 50, pad)
    between = {dt: torch.ones_like(f, dtype=torch.bool) for dt, f in flats.items()}
    for t in g:
        between[t.dtype][t.storage_offset():t.storage_offset() + t.numel()] = False
    obefore = {dt: f.clone() for dt, f in oflats.items()}
    n2 = moe.moe_clip_grad_norm(g, max_norm, out=o)
    assert torch.equal(n, n2)
    _check(o, src, norm, max_norm)
    for dt, f in flats.items():
        assert torch.equal(f, before[dt])                       # the gradients stay
        assert torch.equal(oflats[dt][between[dt]], obefore[dt][between[dt]])
    moe.moe_clip_grad_norm(g, max_norm)
    for a, b in zip(g, o):
        assert torch.equal(a, b)
    for dt, f in flats.items():
        assert torch.equal(f[between[dt]], before[dt][between[dt]])
    for a, b in zip(g, src):
        a.copy_(b)
    moe.moe_grad_clip(g, n, max_norm)
    _check(g, src, norm, max_norm)
    if max_norm == 1e6:
        for a, b in zip(g, src):
            assert torch.equal(a, b)


def test_other_places_of_out():
    """Out tensors at other alignments than the gradients."""
    g, _ = _tensors([5000, 40001, 9], [F32, BF16, BF16], 9, 1)
    o, _ = _tensors([5000, 40001, 9], [F32, BF16, BF16], 10, 2)
    n = moe.moe_clip_grad_norm(g, 1.0, out=o)
    _check(o, g, _norm64(g), 1.0)


@pytest.mark.parametrize("count", [1, 63, 64, 65, 200])
def test_many_tensors(count):
    """Lists of more tensors than a launch takes, empty ones among them."""
    rng = np.random.default_rng(count)
    sizes = [0 if i % 17 == 5 else int(rng.integers(1, 20000)) for i in range(count)]
    dts = [F32 if i % 2 else BF16 for i in range(count)]
    g, _ = _tensors(sizes, dts, 11, 1)
    src = [t.clone() for t in g]
    norm = _norm64(g)
    assert abs(float(moe.moe_grad_norm(g)) - norm) <= 2 * U * norm
    n = moe.moe_clip_grad_norm(g, 2.0)
    assert abs(float(n) - norm) <= 2 * U * norm
    _check(g, src, norm, 2.0)


@pytest.mark.parametrize("sizes", [
    [1], [64], [1023, 1], [16384], [16385], [1024] * 16, [1024] * 15 + [1025], [1] * 16, [1] * 17,
    [0, 5000, 0, 1025, 0, 0, 3, 4096, 0], [2, 16000], [0] * 70 + [900, 65] + [0] * 30])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_short_lists(sizes, kind):
    """Up to 16 pieces of 1024 elements take one launch, more of them several:
    the norm, in place, into other tensors and by a given norm."""
    dts = [{"f32": F32, "bf16": BF16}.get(kind) or (F32 if i % 2 else BF16) for i in range(len(sizes))]
    for pad in (0, 1):
        g, flats = _tensors(sizes, dts, 21, pad)
        src, before = [t.clone() for t in g], {dt: f.clone() for dt, f in flats.items()}
        o, oflats = _tensors(sizes, dts, 22, pad)
        norm = _norm64(g)
        n = moe.moe_grad_norm(g)
        assert abs(float(n) - norm) <= 2 * U * norm
        assert torch.equal(moe.moe_clip_grad_norm(g, 0.25, out=o), n)
        _check(o, src, norm, 0.25)
        assert all(torch.equal(f, before[dt]) for dt, f in flats.items())
        assert torch.equal(moe.moe_clip_grad_norm(g, 0.25), n)
        assert all(torch.equal(a, b) for a, b in zip(g, o))
        for t, b in zip(g, src):
            t.copy_(b)
        assert all(torch.equal(f, before[dt]) for dt, f in flats.items())   # between them
        moe.moe_grad_clip(g, n, 0.25)
        _check(g, src, norm, 0.25)


def test_all_empty():
    e = torch.empty(0, device="cuda")
    assert float(moe.moe_grad_norm([e, e])) == 0.0
    assert float(moe.moe_clip_grad_norm([e], 1.0)) == 0.0
    moe.moe_grad_clip([e], torch.ones((), device="cuda"), 1.0)


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-44])
def test_range(value):
    """Values whose squares leave fp32's range, a norm that leaves it or not."""
    g = torch.full((70000,), value, device="cuda")
    g[::3] *= -0.5
    v = g.cpu().numpy().astype(np.float64)
    norm = math.sqrt((v * v).sum())
    n = float(moe.moe_grad_norm([g]))
    if norm < 3.4e38:
        assert abs(n - norm) <= 2 * U * norm + 2.0 ** -150
        src = g.clone()
        moe.moe_clip_grad_norm([g], 1.0)
        _check([g], [src], norm, 1.0)
    else:
        assert n == math.inf


@pytest.mark.parametrize("dt", [F32, BF16])
def test_nan_and_infinity(dt):
    """An infinity: factor 0, NaN where it is; a NaN: everything is one."""
    g = dev(synth.normal((10000,), 13, 0, 1.0), dt)
    for bad in (math.inf, -math.inf):
        a = g.clone()
        a[77] = bad
        assert float(moe.moe_clip_grad_norm([a], 1.0)) == math.inf
        assert torch.isnan(a[77]) and int((a == 0).sum()) == a.numel() - 1
    a = g.clone()
    a[9999] = math.nan
    b = g.clone()
    assert math.isnan(float(moe.moe_clip_grad_norm([b, a], 1.0)))
    assert torch.isnan(a).all() and torch.isnan(b).all()


def test_factor_of_one_leaves_the_bits():
    g = dev(synth.normal((5000,), 14, 0, 1e-3), F32)
    g[3] = -0.0
    old = g.clone()
    moe.moe_clip_grad_norm([g], 1.0)
    assert torch.equal(g.view(torch.int32), old.view(torch.int32))


def test_element_count_past_32_bits():
    """A tensor of more than 2^31 elements and 2^32 bytes."""
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-3:] = 2.0
    g[0] = 1.0
    g[1 << 31] = 4.0
    want = math.sqrt(12 + 1 + 16)
    assert abs(float(moe.moe_grad_norm([g])) - want) <= 2 * U * want
    moe.moe_clip_grad_norm([g], 1.0)
    s = 1 / (want + 1e-6)
    for i, v in ((0, 1.0), (1 << 31, 4.0), (n - 1, 2.0), (n - 3, 2.0)):
        assert abs(float(g[i]) - v * s) <= v * s * (2.0 ** -8 + 2 * U)
    assert int((g != 0).sum()) == 5


def test_same_bits_every_time():
    g, _ = _tensors([3000000, 777, 123457], [F32, BF16, BF16], 15, 1)
    a = moe.moe_grad_norm(g)
    for _ in range(3):
        assert torch.equal(a, moe.moe_grad_norm(g))


def test_captured_replays_and_streams():
    """Captured on a side stream, replayed on new gradients with eager calls
    in between (their own workspaces): every replay clips by its own norm."""
    g, flats = _tensors([300000, 5, 70001], [F32, F32, BF16], 16, 1)
    o = [torch.empty_like(t) for t in g]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        moe.moe_clip_grad_norm(g, 1.0, out=o)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = moe.moe_clip_grad_norm(g, 1.0, out=o)
    for i in range(3):
        for f in flats.values():
            f.mul_(1.5 if i else 1e-6)
        graph.replay()
        m = moe.moe_grad_norm(g)
        torch.cuda.synchronize()
        norm = _norm64(g)
        assert torch.equal(n, m) and abs(float(n) - norm) <= 2 * U * norm
        _check(o, g, norm, 1.0)


def test_a_training_step_of_two_layers():
    """The weight gradients of two layers and of the norm between them,
    accumulated over two micro-batches, clipped together in place: the next
    accumulation goes on from the clipped ones."""
    T, d, E, k, h = 130, 64, 4, 2, 32
    r = lambda s, i, c=1.0: synth.normal(s, 23, i, c)
    norm = moe.RMSNorm(dev(1 + r((d,), 0, 0.1), F32))
    layers = [moe.MoELayer(dev(r((E, 2 * h, d), 1 + i, 0.1), F32), dev(r((E, d, h), 3 + i, 0.1), F32), k)
              for i in range(2)]
    for mb in range(2):
        x, dout = dev(r((T, d), 10 + mb), F32), dev(r((T, d), 12 + mb), F32)
        logits = [dev(r((T, E), 14 + 2 * mb + i), F32) for i in range(2)]
        a = layers[0].forward(x, logits[0])
        out = layers[1].forward(norm.forward(a, x), logits[1])
        g1 = layers[1].backward(dout, accumulate_dw=mb > 0)
        gn = norm.backward(g1["dx"], dout, accumulate_dw=mb > 0)
        g0 = layers[0].backward(gn["dx"], accumulate_dw=mb > 0)
    grads = [g0["dw1"], g0["dw2"], gn["dweight"], g1["dw1"], g1["dw2"]]
    src = [t.clone() for t in grads]
    n = moe.moe_clip_grad_norm(grads, 0.25)
    _check(grads, src, _norm64(src), 0.25)
    clipped = g0["dw2"].clone()
    layers[0].backward(gn["dx"], accumulate_dw=True)
    fresh = moe.MoELayer(layers[0].w1, layers[0].w2, k)
    fresh.forward(x, logits[0])
    want = clipped + fresh.backward(gn["dx"])["dw2"]
    assert torch.equal(g0["dw2"], want)


def test_refusals():
    g = dev(synth.normal((64, 8), 17, 0, 1.0), F32)
    with pytest.raises(ValueError, match=r"grads\[1\]: expected a contiguous"):
        moe.moe_grad_norm([g, g[:, ::2]])
    with pytest.raises(ValueError, match=r"grads\[0\]: expected a contiguous"):
        moe.moe_grad_norm([g.half()])
    with pytest.raises(ValueError, match=r"out\[0\]"):
        moe.moe_clip_grad_norm([g], 1.0, out=[g.bfloat16()])
    with pytest.raises(ValueError, match="norm"):
        moe.moe_grad_clip([g], torch.ones(2, device="cuda"), 1.0)
    with pytest.raises(ValueError, match="ws"):
        moe.moe_grad_norm([g], ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for bad in ([g, g], [g, g.view(-1)[5:9]]):
        with pytest.raises(moe.MoeError, match="SHAPE"):
            moe.moe_clip_grad_norm(bad, 1.0)
    two = moe.moe_grad_norm([g, g])                       # read only: counts twice
    want = math.sqrt(2) * _norm64([g])
    assert abs(float(two) - want) <= 2 * U * want


# One launch; few partial sums; more partial sums than workgroups (a launch of 64
# such tensors has 2368 chunks).
LENGTHS = {"short": [900, 65], "one tensor": [70000], "few sums": [8192 * 5 + 1] * 70, "many sums": [300000] * 130}


@pytest.mark.parametrize("sizes", LENGTHS.values(), ids=LENGTHS)
def test_the_factor_is_rounded_once(sizes):
    """Whole numbers, whose squares' sum fp64 holds: the factor is the 64-bit
    norm's, rounded to fp32, whatever the list's length (max_norm is one for which
    the norm's own rounding would show), and an fp32 product's one rounding gives
    every bit. moe_grad_clip takes the norm as fp32 holds it."""
    g, _ = _tensors(sizes, [F32] * len(sizes), 31, 1)
    for t in g:
        t.mul_(50).round_()
    norm = math.sqrt(sum(int((t.double() ** 2).sum()) for t in g))
    rounded = float(np.float32(norm))
    factor = lambda n, m: np.float32(float(np.float32(m)) / (n + 1e-6))
    max_norm = next(m / 64 for m in range(1, 512) if factor(norm, m / 64) != factor(rounded, m / 64))
    want = [to_np(t) * factor(norm, max_norm) for t in g]
    given = [to_np(t) * factor(rounded, max_norm) for t in g]
    o = [torch.empty_like(t) for t in g]
    n = moe.moe_clip_grad_norm(g, max_norm, out=o)
    assert float(n) == rounded
    assert all(np.array_equal(to_np(a), b) for a, b in zip(o, want))
    moe.moe_grad_clip(g, n, max_norm, out=o)
    assert all(np.array_equal(to_np(a), b) for a, b in zip(o, given))
    moe.moe_clip_grad_norm(g, max_norm)
    assert all(np.array_equal(to_np(a), b) for a, b in zip(g, want))


@pytest.mark.parametrize("max_norm", [0.0, 1.0, 3e38, math.inf])
@pytest.mark.parametrize("sizes", LENGTHS.values(), ids=LENGTHS)
def test_a_norm_past_fp32(sizes, max_norm):
    """Finite gradients with a norm beyond fp32's range: the norm is infinite and
    the factor 0, in lists of every length, in place and not, and by that norm."""
    g = [torch.full((s,), 3e38, device="cuda") for s in sizes]
    for t in g:
        t[::2] *= -1
    o = [torch.ones_like(t) for t in g]
    n = moe.moe_clip_grad_norm(g, max_norm, out=o)
    assert float(n) == math.inf and float(moe.moe_grad_norm(g)) == math.inf
    assert all((t == 0).all() for t in o)
    p = [torch.ones_like(t) for t in g]
    moe.moe_grad_clip(g, n, max_norm, out=p)
    assert all((t == 0).all() for t in p)
    moe.moe_clip_grad_norm(g, max_norm)
    assert all((t == 0).all() for t in g)
