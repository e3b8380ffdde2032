"""The root-mean-square norm on the GPU against the plain 64-bit form, and its
8-bit output against the quantiser.

Tolerances count roundings, u = 2^-24 each and h = half a step of the stored
type relative to the value. A row's sum adds at most 64 + 10 times per term (64
elements a thread, 6 steps in a wave, 3 over waves): n = 75 roundings of the
magnitudes' sum.
  rstd   the sum of squares n + 3 roundings (all terms positive), halved by the
         root, and the root's, the division's and eps's own: 45 u
  y      s rstd gamma: rstd's 45 u and two products: 48 u |y| + h |y|
  dx     with rstd given: xh u; the mean n + 4 roundings:
         4 u r |g| + (n + 8) u r |xh| mean|g xh|, + (h + 2 u) |dx|
  dgamma a sum over T rows in some order: (T + 8) u sum|dy xh|"""
import numpy as np
import pytest
import torch

import oracle
import oracle.train_ops as ops
import synth
from helpers import dev, to_np

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
U = 2.0 ** -24
N = 75
EPS = 1e-6
SHAPES = [(1, 32), (2, 96), (37, 160), (5, 256), (33, 288), (70, 512), (3, 1056), (65, 2048), (1, 2048),
          (9, 2080), (4, 4128), (7, 8192), (2, 8224), (3, 16384)]


def _f64(t):
    return to_np(t).astype(np.float64)


def _near(got, ref, tol, what):
    got, ref, tol = (np.asarray(a, np.float64) for a in (got, ref, tol))
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) / tol)))


def _inputs(T, d, dt, seed):
    rng = np.random.default_rng(seed)
    ch = np.exp(0.5 * rng.normal(size=d)).astype(np.float32)
    x = dev(synth.normal((T, d), seed, 0, 1.0) * ch, DT[dt])
    r = dev(synth.normal((T, d), seed, 1, 1.0), DT[dt])
    ga = torch.from_numpy((1 + 0.1 * rng.normal(size=d)).astype(np.float32)).cuda()
    return x, r, ga


def _check_forward(out, s, ga, dt, what):
    y, rstd = ops.rms_norm(s, _f64(ga), EPS)
    if "rstd" in out:
        _near(_f64(out["rstd"]), rstd, 45 * U * rstd, what + " rstd")
    if "y" in out:
        _near(_f64(out["y"]), y, (48 * U + H[dt]) * np.abs(y) + 2.0 ** -126, what + " y")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(dt, T, d):
    x, r, ga = _inputs(T, d, dt, T + d)
    for res in (None, r):
        for act8 in (False, True):
            what = f"res {res is not None} act8 {act8}"
            out = moe.moe_rms_norm(x, ga, EPS, residual=res, quantize=True, act8=act8)
            s = _f64(x)
            if res is not None:
                want = (x.float() + res.float()).to(DT[dt])
                assert torch.equal(out["sum"], want), what
                s = _f64(want)
            _check_forward(out, s, ga, dt, what)
            q, e = moe.mxfp8_quantize(out["y"], 1)
            assert torch.equal(out["yq"], q) and torch.equal(out["yq_scale"], e), what
            q, e = oracle.mxfp8_quantize(to_np(out["y"]), 1)
            assert np.array_equal(to_np(out["yq"]).ravel(), np.asarray(q).ravel()), what
            assert np.array_equal(to_np(out["yq_scale"]).ravel(), np.asarray(e).ravel()), what
            if act8:
                c, e = ops.act8_encode(s)
                assert np.array_equal(to_np(out["x8"]).view(np.int8), c), what
                assert np.array_equal(to_np(out["x8_scale"]), e), what
            only = moe.moe_rms_norm(x, ga, EPS, residual=res, quantize=True, want_y=False, stats=False)
            assert set(only) == {"yq", "yq_scale"} | ({"sum"} if res is not None else set())
            assert torch.equal(only["yq"], out["yq"]) and torch.equal(only["yq_scale"], out["yq_scale"])
            lean = moe.moe_rms_norm(x, ga, EPS, residual=res, stats=False)
            assert torch.equal(lean["y"], out["y"]) and "yq" not in lean


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 160, 288, 512, 2048, 2080, 4128, 8224, 16384])
def test_rounded_once(dt, d):
    """Whole numbers up to 8, whose squares' sum (at most 2^20) fp32 holds: rstd
    is then known to 2^-46, s rstd gamma to 2^-45 or better, and rounded to fp32
    it is the 64-bit value's rounding but for one element in 2^20 (those that lie
    so close to the middle of two fp32 numbers). None may differ in bf16."""
    rng = np.random.default_rng(d)
    T = 37
    s = rng.integers(-8, 9, (T, d)).astype(np.float64)
    ga = (1 + 0.1 * rng.normal(size=d)).astype(np.float32)
    out = moe.moe_rms_norm(dev(s, DT[dt]), torch.from_numpy(ga).cuda(), EPS)
    y, rstd = ops.rms_norm(s, ga.astype(np.float64), float(np.float32(EPS)))
    want = torch.from_numpy(y.astype(np.float32)).to(DT[dt])
    diff = int((out["y"].cpu() != want).sum())
    assert diff <= (1 if dt == "f32" else 0), diff
    assert np.array_equal(to_np(out["rstd"]), np.asarray(rstd, np.float64).astype(np.float32).ravel())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gamma", [np.inf, -np.inf, 3e38, 1e-45])
def test_extreme_weights(dt, gamma):
    """A weight beyond the values' range: the formula's infinities, zeros and
    NaNs (of a zero times an infinity), nothing else."""
    s = np.array([[1.0, -2.0, 0.0, 3.0] * 16, [0.0] * 64, [1e-3, -1e3, 5.0, 0.25] * 16])
    ga = np.ones(64, np.float32)
    ga[::3] = gamma
    out = moe.moe_rms_norm(dev(s, DT[dt]), torch.from_numpy(ga).cuda(), EPS)
    x = dev(s, DT[dt]).double().cpu()
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    want = (x * r * torch.from_numpy(ga).double()).float().to(DT[dt])
    got = out["y"].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    ok = torch.isfinite(want)
    d = (got.double() - want.double()).abs()[ok]
    # half a step of each side's rounding, and fp32's
    assert (d <= want.double().abs()[ok] * (2 * H[dt] + 48 * U) + 2.0 ** -133).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 1024, 4096])
def test_forward_hard_rows(dt, d):
    """Constant rows, zeros, tiny and huge ones, an outlier; a NaN or an
    infinity spoils no other row."""
    x = synth.normal((9, d), 7, 0, 1.0)
    x[0], x[1] = 3.0, 0.0
    x[2] += 4096.0
    x[3] *= 1e-18
    x[4] *= 1e15
    x[5, 0] = 1e4                                           # one outlier
    t = dev(x, DT[dt])
    ga = torch.full((d,), 1.5, device="cuda")
    out = moe.moe_rms_norm(t, ga, EPS, quantize=True)
    _check_forward(out, _f64(t), ga, dt, "hard")
    assert (out["y"][1] == 0).all() and (out["yq"][1] == 0).all() and (out["yq_scale"][1] == 0).all()
    bad = t.clone()
    bad[6, d // 2], bad[8, 1] = float("nan"), float("inf")
    o2 = moe.moe_rms_norm(bad, ga, EPS, quantize=True)
    keep = [0, 1, 2, 3, 4, 5, 7]
    for n in ("y", "rstd", "yq", "yq_scale"):
        assert torch.equal(o2[n][keep], out[n][keep]), n
    assert torch.isnan(o2["y"][6]).all()
    assert o2["rstd"][8] == 0 and torch.isnan(o2["y"][8, 1]) and (o2["y"][8, 2:] == 0).all()
    q, e = moe.mxfp8_quantize(o2["y"], 1)
    assert torch.equal(o2["yq"], q) and torch.equal(o2["yq_scale"], e)


def _check_backward(b, s, rstd, dy, ga, ds, dt, T, what):
    dyf, g, r = _f64(dy), _f64(dy) * _f64(ga), rstd[:, None]
    dx, dg = ops.rms_norm_backward(s, rstd, dyf, _f64(ga), None if ds is None else _f64(ds))
    xh = s * r
    tol = r * U * (4 * np.abs(g) + (N + 8) * np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    _near(_f64(b["dx"]), dx, tol + (H[dt] + 2 * U) * np.abs(dx) + 2.0 ** -126, what + " dx")
    if "dweight" in b:
        _near(_f64(b["dweight"]), dg, (T + 8) * U * np.abs(dyf * xh).sum(0) + 1e-30, what + " dweight")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES + [(3000, 32), (2200, 544), (700, 4096)])
def test_backward(dt, T, d):
    """From x and from its checkpoint, with and without a stream gradient;
    the last sizes give every workgroup several rows."""
    x, ds, ga = _inputs(T, d, dt, T + d + 1)
    dy = dev(synth.normal((T, d), 8, 2, 1.0), DT[dt])
    f = moe.moe_rms_norm(x, ga, EPS, act8=True)
    val = ops.act8_decode(to_np(f["x8"]).view(np.int8), to_np(f["x8_scale"]))
    for src, s in ((dict(f, x=x), _f64(x)), (f, val)):
        for dsum in (None, ds):
            what = f"x {'x' in src} dsum {dsum is not None}"
            b = moe.moe_rms_norm_backward(src, dy, ga, dsum)
            _check_backward(b, s, _f64(f["rstd"]), dy, ga, dsum, dt, T, what)
            only = moe.moe_rms_norm_backward(src, dy, ga, dsum, want_dweight=False)
            assert set(only) == {"dx"} and torch.equal(only["dx"], b["dx"])
            old = {n: v.clone() for n, v in b.items()}
            moe.moe_rms_norm_backward(src, dy, ga, dsum, out=b, accumulate_dw=True)
            assert torch.equal(b["dweight"], old["dweight"] + old["dweight"])
            assert torch.equal(b["dx"], old["dx"])


def test_backward_by_differences():
    """The kernel's fp32 gradient along directions against central differences
    of the 64-bit forward: O(h^2) = 1e-8 of O(1) third derivatives, and the
    gradient's own fp32 roundings (1e-6 of the terms' sum)."""
    T, d = 6, 96
    x, ds, ga = _inputs(T, d, "f32", 11)
    dy = dev(synth.normal((T, d), 11, 2, 1.0), torch.float32)
    f = moe.moe_rms_norm(x, ga, EPS)
    b = moe.moe_rms_norm_backward(dict(f, x=x), dy, ga, ds)
    s, g = _f64(x), _f64(ga)
    loss = lambda a, w: (ops.rms_norm(a, w, EPS)[0] * _f64(dy)).sum() + (a * _f64(ds)).sum()
    rng, h = np.random.default_rng(3), 1e-4
    for _ in range(5):
        vx, vg = rng.normal(size=(T, d)), rng.normal(size=d)
        num = (loss(s + h * vx, g + h * vg) - loss(s - h * vx, g - h * vg)) / (2 * h)
        terms = [(_f64(b["dx"]) * vx).ravel(), _f64(b["dweight"]) * vg]
        assert abs(num - sum(t.sum() for t in terms)) <= 1e-6 * sum(np.abs(t).sum() for t in terms)


def test_no_rows():
    ga = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    f = moe.moe_rms_norm(e, ga, quantize=True, act8=True)
    assert f["y"].shape == (0, 64) and f["yq"].shape == (0, 64)
    b = moe.moe_rms_norm_backward(dict(f, x=e), e, ga)
    assert (b["dweight"] == 0).all()
    b["dweight"].fill_(3)
    moe.moe_rms_norm_backward(dict(f, x=e), e, ga, out=b, accumulate_dw=True)
    assert (b["dweight"] == 3).all()


@pytest.mark.parametrize("T,d", [(3, 160), (5, 2080), (2, 8224)])
def test_nothing_else_is_written(T, d):
    """Outputs inside larger buffers; the buffers' ends stay as they were."""
    x, r, ga = _inputs(T, d, "bf16", 5)
    big = lambda n, dt, v: torch.full((n,), v, dtype=dt, device="cuda")
    n = T * d
    bufs = dict(y=big(n + 16, torch.bfloat16, 9), sum=big(n + 16, torch.bfloat16, 9),
                rstd=big(T + 16, torch.float32, 9), yq=big(n + 16, torch.uint8, 9),
                yq_scale=big(n // 32 + 16, torch.uint8, 9))
    view = dict(y=bufs["y"][:n].view(T, d), sum=bufs["sum"][:n].view(T, d), rstd=bufs["rstd"][:T],
                yq=bufs["yq"][:n].view(T, d), yq_scale=bufs["yq_scale"][:n // 32].view(T, d // 32))
    moe.moe_rms_norm(x, ga, EPS, residual=r, quantize=True, out=view)
    for k, v in bufs.items():
        assert (v[-16:] == 9).all(), k
    g = dict(dx=big(n + 16, torch.bfloat16, 9), dweight=big(d + 16, torch.float32, 9))
    wsb = moe.moe_rms_norm_backward_workspace_size(moe.MOE_BF16, T, d)
    ws = big(wsb + 16, torch.uint8, 9)
    moe.moe_rms_norm_backward(dict(rstd=view["rstd"], x=x), r, ga, x, ws=ws[:wsb],
                              out=dict(dx=g["dx"][:n].view(T, d), dweight=g["dweight"][:d]))
    for k, v in dict(g, ws=ws).items():
        assert (v[-16:] == 9).all(), k


def test_offsets_past_32_bits():
    """More rows than one launch takes and more than 2^32 bytes: the last rows
    come out as they do by themselves."""
    d, T = 2080, (1 << 21) + 5                             # 2^21 workgroups of one row a launch
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    x.fill_(1)
    tail = torch.randn(6, d, device="cuda").bfloat16()
    x[-6:] = tail
    ga = torch.ones(d, device="cuda")
    f = moe.moe_rms_norm(x, ga, quantize=True)
    one = moe.moe_rms_norm(tail, ga, quantize=True)
    for k in ("y", "rstd", "yq", "yq_scale"):
        assert torch.equal(f[k][-6:], one[k]), k
    v = moe.mxfp8_dequantize(f["yq"], f["yq_scale"])
    assert torch.equal(v[-6:], moe.mxfp8_dequantize(one["yq"], one["yq_scale"]))
    b = moe.moe_rms_norm_backward(dict(f, x=x), x, ga, out=dict(
        dx=f["y"], dweight=torch.empty(d, device="cuda")))
    b1 = moe.moe_rms_norm_backward(dict(one, x=tail), tail, ga)
    assert torch.equal(b["dx"][-6:], b1["dx"])


@pytest.mark.parametrize("dt,T,d", [("bf16", 8200, 4096), ("f32", 4100, 4128), ("bf16", 33000, 1056)])
@pytest.mark.parametrize("act8", [False, True])
def test_backward_of_large_matrices(dt, T, d, act8):
    """Matrices beyond what the last-level cache is used for (their kernel is
    one of its own, whose roundings may fall elsewhere): the formula."""
    x, ds, ga = _inputs(T, d, dt, 5)
    dy = dev(synth.normal((T, d), 9, 2, 1.0), DT[dt])
    f = moe.moe_rms_norm(x, ga, EPS, act8=act8)
    b = moe.moe_rms_norm_backward(f if act8 else dict(f, x=x), dy, ga, ds)
    s = ops.act8_decode(to_np(f["x8"]).view(np.int8), to_np(f["x8_scale"])) if act8 else _f64(x)
    _check_backward(b, s, _f64(f["rstd"]), dy, ga, ds, dt, T, "large")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dequantize_every_code(dt):
    """Every element under every scale byte: exact in fp32, rounded once in
    bf16; scale byte 255 stands for NaNs."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()         # [256 scales, 256 codes]
    e = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8).cuda()
    got = moe.mxfp8_dequantize(q, e, DT[dt])
    table = np.asarray(oracle.e4m3_decode_table(), np.float64).reshape(1, 256)
    want = table * np.exp2(np.arange(256, dtype=np.float64) - 127)[:, None]
    want = torch.from_numpy(want).to(torch.float32)                        # exact: 4 bits over 2^-136
    want[255] = float("nan")
    want = want.to(DT[dt])
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(0, 64), (1, 32), (3, 96), (77, 352), (129, 4096)])
def test_dequantize_what_was_quantised(dt, rows, cols):
    x = dev(synth.normal((rows, cols), 3, 0, 2.0), DT[dt])
    q, e = moe.mxfp8_quantize(x, 1) if rows else (torch.empty(0, cols, dtype=torch.uint8, device="cuda"),
                                                  torch.empty(0, cols // 32, dtype=torch.uint8, device="cuda"))
    out = torch.full((rows * cols + 16,), 9.0, dtype=DT[dt], device="cuda")
    got = moe.mxfp8_dequantize(q, e, DT[dt], out=out[:rows * cols].view(rows, cols))
    assert (out[rows * cols:] == 9).all()
    if rows:
        want = oracle.mxfp8_dequantize_rowwise(to_np(q), to_np(e))
        assert np.array_equal(_f64(got), np.asarray(want, np.float64))


@pytest.mark.parametrize("recompute", [False, True])
def test_norm_feeds_the_mxfp8_layer(recompute):
    """The 8-bit rows that the norm writes are those that the layer would make
    of y: the same output and gradients, bit for bit; and the chain's gradient
    through the norm follows its formula."""
    T, d, E, k, h = 300, 256, 8, 2, 128
    n = lambda s, i, c=1.0: synth.normal(s, 21, i, c)
    w1, w2 = dev(n((E, 2 * h, d), 0, 0.05), torch.float32), dev(n((E, d, h), 1, 0.05), torch.float32)
    x, res = dev(n((T, d), 2), torch.bfloat16), dev(n((T, d), 3), torch.bfloat16)
    wr, ga = dev(n((E, d), 4, 0.1), torch.float32), dev(1 + n((d,), 5, 0.1), torch.float32)
    dout = dev(n((T, d), 6), torch.bfloat16)
    norm = moe.RMSNorm(ga, quantize=True)
    plain, fed = (moe.MoELayerMX(w1, w2, k, recompute=recompute) for _ in range(2))
    y = norm.forward(x, res)
    logits = y.float() @ wr.t()
    a = plain.forward(y, logits).clone()
    b = fed.forward(y, logits, xq=norm.q)
    assert torch.equal(a, b)
    ga_, gb_ = plain.backward(dout), fed.backward(dout)
    for name in ("dx", "dlogits", "dw1", "dw2"):
        assert torch.equal(ga_[name], gb_[name]), name
    dy = (gb_["dx"].float() + gb_["dlogits"] @ wr).to(torch.bfloat16)
    g = norm.backward(dy, dout)
    _check_backward(g, _f64(norm.sum), _f64(norm._out["rstd"]), dy, ga, dout, "bf16", T, "chain")
    with pytest.raises(ValueError, match="xq"):
        fed.forward(y, logits, xq=(norm.q[0][:-1], norm.q[1]))


def test_as_out_norm():
    """Behind the layer: the layer's backward goes through it and reports its
    weight's gradient (there is no bias)."""
    T, d, E, k, h = 65, 64, 4, 2, 32
    n = lambda s, i, c=1.0: synth.normal(s, 22, i, c)
    w1, w2 = dev(n((E, 2 * h, d), 0, 0.1), torch.float32), dev(n((E, d, h), 1, 0.1), torch.float32)
    x, logits = dev(n((T, d), 2), torch.float32), dev(n((T, E), 3), torch.float32)
    ga, dout = dev(1 + n((d,), 4, 0.1), torch.float32), dev(n((T, d), 5), torch.float32)
    norm = moe.RMSNorm(ga)
    layer = moe.MoELayer(w1, w2, k, out_norm=norm)
    out = layer.forward(x, logits)
    f = moe.moe_rms_norm(layer.out, ga)
    assert torch.equal(out, f["y"])
    g = layer.backward(dout)
    want = moe.moe_rms_norm_backward(dict(f, x=layer.out), dout, ga)
    assert torch.equal(g["dnorm_weight"], want["dweight"]) and g["dnorm_bias"] is None
    ref = moe.MoELayer(w1, w2, k)
    ref.forward(x, logits)
    assert torch.equal(ref.backward(want["dx"])["dx"], g["dx"])


def test_captured_replays():
    """Forward and backward in a graph, replayed on new inputs between eager
    work: every replay gives the eager result."""
    T, d = 70, 1024
    x, r, ga = _inputs(T, d, "bf16", 31)
    norm = moe.RMSNorm(ga, quantize=True, act8=True)
    dy = dev(synth.normal((T, d), 31, 4, 1.0), torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm.forward(x, r)
        norm.backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = norm.forward(x, r)
        g = norm.backward(dy)
    q = norm.q
    for i in range(3):
        x.copy_(dev(synth.normal((T, d), 32, i, 1.0), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        f = moe.moe_rms_norm(x, ga, residual=r, quantize=True, act8=True)
        b = moe.moe_rms_norm_backward(f, dy, ga)
        for got, want in ((y, f["y"]), (q[0], f["yq"]), (q[1], f["yq_scale"]), (g["dx"], b["dx"]),
                          (g["dweight"], b["dweight"])):
            assert torch.equal(got, want), i


def test_refused_calls_leave_the_object_usable():
    n = lambda i, t: dev(synth.normal((t, 256), 41, i, 1.0), torch.float32)
    w = dev(1 + synth.normal((256,), 41, 9, 0.1), torch.float32)
    norm = moe.RMSNorm(w)
    with pytest.raises(ValueError, match="without a forward"):
        norm.backward(n(2, 300))
    norm.forward(n(1, 300))
    with pytest.raises(ValueError, match="x: expected"):
        norm.backward(n(2, 3))
    with pytest.raises(ValueError, match="residual"):
        norm.forward(n(1, 8), n(3, 9))
    with pytest.raises(ValueError, match="without a forward"):
        norm.backward(n(2, 8))
    norm.forward(n(1, 8), n(3, 8))
    f = moe.moe_rms_norm(n(1, 8) + n(3, 8), w)
    want = moe.moe_rms_norm_backward(dict(f, x=n(1, 8) + n(3, 8)), n(2, 8), w)["dx"]
    assert torch.equal(norm.backward(n(2, 8))["dx"], want)
    with pytest.raises(ValueError, match="want_y"):
        moe.moe_rms_norm(n(1, 8), w, want_y=False)


def test_an_objects_outputs_may_change():
    """quantize and act8 set and taken back between two forwards of a size."""
    x = dev(synth.normal((33, 96), 31, 0, 1.0), torch.bfloat16)
    norm = moe.RMSNorm(dev(synth.normal((96,), 31, 1, 1.0), torch.float32))
    y = norm.forward(x).clone()
    assert norm.q is None
    norm.quantize = True
    assert torch.equal(norm.forward(x), y)
    q, s = moe.mxfp8_quantize(y, 1)
    assert torch.equal(norm.q[0].view(-1), q.view(-1)) and torch.equal(norm.q[1].view(-1), s.view(-1))
    norm.act8 = True
    assert torch.equal(norm.forward(x), y)
    norm.backward(y)
    norm.quantize = norm.act8 = False
    assert torch.equal(norm.forward(x), y) and norm.q is None
    norm.backward(y)
