"""The layer norm on the GPU against the plain 64-bit form.

Tolerances count roundings, u = 2^-24 each and h = half a step of the stored
type relative to the value (2^-8 for bf16's 8 significant bits, u for fp32). A
row's sum adds at most 64 + 10 times per term (64 elements a thread, 6 steps
in a wave, 3 over waves): n = 75 roundings of the magnitudes' sum.
  mean   n u mean|s|
  rstd   the variance n + 4 roundings (the mean's error is of second order in
         it, (n u mean|s|)^2), the root halves them: 45 u, and eps's share
  y      r |gamma| n u mean|s| + 50 u |xh gamma| + 3 u |y| + h |y|
  dx     with the statistics given: xh 2 u; the two means n + 4 roundings;
         4 u r |g| + (n + 8) u r (mean|g| + |xh| mean|g xh|), + h |dx|
  dgamma a sum over T rows in some order: (T + 8) u sum|dy xh|; dbeta alike"""
import numpy as np
import pytest
import torch

import oracle.train_ops as ops
import synth
from helpers import dev, to_np

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a step: bf16 has 8 significant bits, so steps of 2^-7 in [1, 2) and 2^-8 of the value at most
H = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
U = 2.0 ** -24
N = 75
EPS = 1e-5
SHAPES = [(1, 32), (2, 96), (37, 160), (5, 256), (33, 288), (70, 512), (3, 1056), (65, 2048), (1, 2048),
          (9, 2080), (4, 4128), (7, 8192), (2, 8224), (3, 16384)]


def _f64(t):
    return to_np(t).astype(np.float64)


def _near(got, ref, tol, what):
    got, ref, tol = (np.asarray(a, np.float64) for a in (got, ref, tol))
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) / tol)))


def _inputs(T, d, dt, seed, offset=0.1):
    rng = np.random.default_rng(seed)
    ch = np.exp(0.5 * rng.normal(size=d)).astype(np.float32)
    x = dev(synth.normal((T, d), seed, 0, 1.0) * ch + np.float32(offset), DT[dt])
    r = dev(synth.normal((T, d), seed, 1, 1.0), DT[dt])
    ga = torch.from_numpy((1 + 0.1 * rng.normal(size=d)).astype(np.float32)).cuda()
    be = torch.from_numpy(rng.normal(size=d).astype(np.float32)).cuda()
    return x, r, ga, be


def _check_forward(out, s, ga, be, dt, what):
    g = _f64(ga)
    y, mean, rstd = ops.layer_norm(s, g, None if be is None else _f64(be), EPS)
    ms, xg = np.abs(s).mean(1), np.abs((s - mean[:, None]) * rstd[:, None] * g)
    if "mean" in out:
        _near(_f64(out["mean"]), mean, (N + 2) * U * ms, what + " mean")
        dmu = N * U * ms
        _near(_f64(out["rstd"]), rstd, 45 * U * rstd + rstd ** 3 * dmu ** 2, what + " rstd")
    tol = (rstd[:, None] * np.abs(g) * (N + 2) * U * ms[:, None] + 50 * U * xg
           + (3 * U + H[dt]) * np.abs(y) + 3 * U * (0 if be is None else np.abs(_f64(be)))
           + rstd[:, None] ** 2 * (N * U * ms[:, None]) ** 2 * xg + 2.0 ** -126)
    _near(_f64(out["y"]), y, tol, what + " y")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(dt, T, d):
    x, r, ga, be = _inputs(T, d, dt, T + d)
    for bias in (None, be):
        for res in (None, r):
            for act8 in (False, True):
                what = f"bias {bias is not None} res {res is not None} act8 {act8}"
                out = moe.moe_layer_norm(x, ga, bias, EPS, residual=res, act8=act8)
                s = _f64(x)
                if res is not None:
                    want = (x.float() + res.float()).to(DT[dt])
                    assert torch.equal(out["sum"], want), what
                    s = _f64(want)
                _check_forward(out, s, ga, bias, dt, what)
                if act8:
                    c, e = ops.act8_encode(s)
                    assert np.array_equal(to_np(out["x8"]).view(np.int8), c), what
                    assert np.array_equal(to_np(out["x8_scale"]), e), what
                lean = moe.moe_layer_norm(x, ga, bias, EPS, residual=res, stats=False)
                assert set(lean) == ({"y", "sum"} if res is not None else {"y"})
                assert torch.equal(lean["y"], out["y"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 1024, 4096])
def test_forward_hard_rows(dt, d):
    """Constant rows, rows far from zero, tiny and huge ones, zeros; and rows
    with a NaN or an infinity, which spoil no other row."""
    x = synth.normal((9, d), 7, 0, 1.0)
    x[0], x[1] = 3.0, 0.0
    x[2] += 4096.0
    x[3] *= 1e-18
    x[4] *= 1e15
    x[5, 0] = 1e4                                           # one outlier
    t = dev(x, DT[dt])
    ga, be = torch.full((d,), 1.5, device="cuda"), torch.full((d,), 0.25, device="cuda")
    out = moe.moe_layer_norm(t, ga, be, EPS, act8=True)
    _check_forward(out, _f64(t), ga, be, dt, "hard")
    bad = t.clone()
    bad[6, d // 2], bad[8, 1] = float("nan"), float("inf")
    o2 = moe.moe_layer_norm(bad, ga, be, EPS, act8=True)
    keep = [0, 1, 2, 3, 4, 5, 7]
    for n in ("y", "mean", "rstd", "x8", "x8_scale"):
        assert torch.equal(o2[n][keep], out[n][keep]), n
    assert torch.isnan(o2["y"][6]).all() and torch.isnan(o2["y"][8]).all()
    assert int((o2["x8_scale"] == 255).sum()) == 2


def _check_backward(b, s, st, dy, ga, ds, dt, T, what):
    mean, rstd = _f64(st["mean"]), _f64(st["rstd"])
    dyf, g = _f64(dy), _f64(dy) * _f64(ga)
    dx, dg, db = ops.layer_norm_backward(s, mean, rstd, dyf, _f64(ga), None if ds is None else _f64(ds))
    r = rstd[:, None]
    xh = (s - mean[:, None]) * r
    tol = r * U * (4 * np.abs(g) + (N + 8) * (np.abs(g).mean(1, keepdims=True)
                                              + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True)))
    _near(_f64(b["dx"]), dx, tol + (H[dt] + 2 * U) * np.abs(dx) + 2.0 ** -126, what + " dx")
    if "dweight" in b:
        _near(_f64(b["dweight"]), dg, (T + 8) * U * np.abs(dyf * xh).sum(0) + 1e-30, what + " dweight")
    if "dbias" in b:
        _near(_f64(b["dbias"]), db, (T + 8) * U * np.abs(dyf).sum(0) + 1e-30, what + " dbias")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES + [(3000, 32), (2200, 544), (700, 4096)])
def test_backward(dt, T, d):
    """From x and from its checkpoint, with and without a stream gradient;
    the last sizes give every workgroup several rows."""
    x, ds, ga, _ = _inputs(T, d, dt, T + d + 1)
    dy = dev(synth.normal((T, d), 8, 2, 1.0), DT[dt])
    f = moe.moe_layer_norm(x, ga, None, EPS, act8=True)
    val = ops.act8_decode(to_np(f["x8"]).view(np.int8), to_np(f["x8_scale"]))
    for src, s in ((dict(f, x=x), _f64(x)), (f, val)):
        for dsum in (None, ds):
            what = f"x {'x' in src} dsum {dsum is not None}"
            b = moe.moe_layer_norm_backward(src, dy, ga, dsum)
            _check_backward(b, s, f, dy, ga, dsum, dt, T, what)
            only = moe.moe_layer_norm_backward(src, dy, ga, dsum, want_dweight=False, want_dbias=False)
            assert set(only) == {"dx"} and torch.equal(only["dx"], b["dx"])
            one = moe.moe_layer_norm_backward(src, dy, ga, dsum, want_dbias=False)
            assert set(one) == {"dx", "dweight"} and torch.equal(one["dweight"], b["dweight"])
            old = {n: v.clone() for n, v in b.items()}
            moe.moe_layer_norm_backward(src, dy, ga, dsum, out=b, accumulate_dw=True)
            assert torch.equal(b["dweight"], old["dweight"] + old["dweight"])
            assert torch.equal(b["dbias"], old["dbias"] + old["dbias"]) and torch.equal(b["dx"], old["dx"])


def test_backward_by_differences():
    """The kernel's fp32 gradient along directions against central differences
    of the 64-bit forward: O(h^2) = 1e-8 of O(1) third derivatives, and the
    gradient's own fp32 roundings (1e-6 of the terms' sum)."""
    T, d = 6, 96
    x, ds, ga, be = _inputs(T, d, "f32", 11)
    dy = dev(synth.normal((T, d), 11, 2, 1.0), torch.float32)
    f = moe.moe_layer_norm(x, ga, be, EPS)
    b = moe.moe_layer_norm_backward(dict(f, x=x), dy, ga, ds)
    s, g, c = _f64(x), _f64(ga), _f64(be)
    loss = lambda a, w, v: (ops.layer_norm(a, w, v, EPS)[0] * _f64(dy)).sum() + (a * _f64(ds)).sum()
    rng, h = np.random.default_rng(3), 1e-4
    for _ in range(5):
        vx, vg, vb = rng.normal(size=(T, d)), rng.normal(size=d), rng.normal(size=d)
        num = (loss(s + h * vx, g + h * vg, c + h * vb) - loss(s - h * vx, g - h * vg, c - h * vb)) / (2 * h)
        terms = [(_f64(b["dx"]) * vx).ravel(), _f64(b["dweight"]) * vg, _f64(b["dbias"]) * vb]
        assert abs(num - sum(t.sum() for t in terms)) <= 1e-6 * sum(np.abs(t).sum() for t in terms)


def test_no_rows():
    ga = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    f = moe.moe_layer_norm(e, ga, act8=True)
    assert f["y"].shape == (0, 64)
    b = moe.moe_layer_norm_backward(dict(f, x=e), e, ga)
    assert (b["dweight"] == 0).all() and (b["dbias"] == 0).all()
    b["dweight"].fill_(3)
    moe.moe_layer_norm_backward(dict(f, x=e), e, ga, out=b, accumulate_dw=True)
    assert (b["dweight"] == 3).all()


@pytest.mark.parametrize("T,d", [(3, 160), (5, 2080), (2, 8224)])
def test_nothing_else_is_written(T, d):
    """Outputs inside larger buffers; the buffers' ends stay as they were."""
    x, r, ga, be = _inputs(T, d, "bf16", 5)
    big = lambda n, dt, v: torch.full((n,), v, dtype=dt, device="cuda")
    n = T * d
    bufs = dict(y=big(n + 16, torch.bfloat16, 9), sum=big(n + 16, torch.bfloat16, 9),
                mean=big(T + 16, torch.float32, 9), rstd=big(T + 16, torch.float32, 9),
                x8=big(n + 16, torch.uint8, 9), x8_scale=big(n // 32 + 16, torch.uint8, 9))
    view = dict(y=bufs["y"][:n].view(T, d), sum=bufs["sum"][:n].view(T, d), mean=bufs["mean"][:T],
                rstd=bufs["rstd"][:T], x8=bufs["x8"][:n].view(T, d),
                x8_scale=bufs["x8_scale"][:n // 32].view(T, d // 32))
    moe.moe_layer_norm(x, ga, be, EPS, residual=r, act8=True, out=view)
    for k, v in bufs.items():
        assert (v[-16:] == 9).all(), k
    g = dict(dx=big(n + 16, torch.bfloat16, 9), dweight=big(d + 16, torch.float32, 9),
             dbias=big(d + 16, torch.float32, 9))
    wsb = moe.moe_layer_norm_backward_workspace_size(moe.MOE_BF16, T, d)
    ws = big(wsb + 16, torch.uint8, 9)
    moe.moe_layer_norm_backward(view, r, ga, x, ws=ws[:wsb], out=dict(
        dx=g["dx"][:n].view(T, d), dweight=g["dweight"][:d], dbias=g["dbias"][:d]))
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
    f = moe.moe_layer_norm(x, ga, act8=True)
    one = moe.moe_layer_norm(tail, ga, act8=True)
    for k in ("y", "mean", "rstd", "x8", "x8_scale"):
        assert torch.equal(f[k][-6:], one[k]), k
    b = moe.moe_layer_norm_backward(f, x, ga, out=dict(
        dx=f["y"], dweight=torch.empty(d, device="cuda"), dbias=torch.empty(d, device="cuda")))
    b1 = moe.moe_layer_norm_backward(one, tail, ga)
    assert torch.equal(b["dx"][-6:], b1["dx"])
    # constant rows: xh = 0; dbias counts them, in fp32 sums of whole numbers below 2^24
    assert torch.allclose(b["dweight"], b1["dweight"], atol=1e-5)
    assert ((b["dbias"] - (T - 6) - b1["dbias"]).abs() <= 1.0).all()


def test_refused_calls_leave_the_object_usable():
    """A gradient of the wrong size, then a forward that is refused: neither
    leaves buffers of the wrong size or a half-made state behind."""
    n = lambda i, t: dev(synth.normal((t, 256), 41, i, 1.0), torch.float32)
    w = dev(1 + synth.normal((256,), 41, 9, 0.1), torch.float32)
    norm = moe.LayerNorm(w, None, EPS)
    with pytest.raises(ValueError, match="without a forward"):
        norm.backward(n(2, 300))
    norm.forward(n(1, 300))
    with pytest.raises(ValueError, match="x: expected"):
        norm.backward(n(2, 3))
    dx = norm.backward(n(2, 300))["dx"].clone()
    assert torch.equal(dx, _fresh_dx(w, n(1, 300), n(2, 300)))
    with pytest.raises(ValueError, match="residual"):
        norm.forward(n(1, 8), n(3, 9))
    with pytest.raises(ValueError, match="without a forward"):
        norm.backward(n(2, 8))
    norm.forward(n(1, 8), n(3, 8))
    assert torch.equal(norm.backward(n(2, 8))["dx"], _fresh_dx(w, n(1, 8) + n(3, 8), n(2, 8)))


def _fresh_dx(w, x, dy):
    norm = moe.LayerNorm(w, None, EPS)
    norm.forward(x)
    return norm.backward(dy)["dx"]
