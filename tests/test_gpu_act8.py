"""The 8-bit activation checkpoints on the GPU against the plain 64-bit form:
bytes and restored values bit for bit, the operators that read them within
their rounding.

Tolerances count roundings (u = 2^-24, one fp32 rounding; h = half a step of
the stored type relative to the value, 2^-8 for bf16's 8 significant bits and
u for fp32; results below the smallest normal number may be off by half of
the smallest subnormal or flushed):
  H'     silu(a) b: exp takes a few u (at most 4 + |a| with its argument's
         rounding), an add, a quotient, a product: (10 + 2|a|) u + h
  out    k products, k sums: bit-identical to moe_combine
  dgate  a sum of d products over 64 lanes: at most d/64 + 6 additions and a
         product each, of the magnitudes' sum
  dlogits  products and sums of k of these: 4k more roundings"""
import numpy as np
import pytest
import torch

import oracle.train_ops as ops
import synth
from helpers import dev, rel_fro, to_np

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a step: bf16 has 8 significant bits, so steps of 2^-7 in [1, 2) and 2^-8 of the value at most
H = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
U = 2.0 ** -24


def _values(rows, cols, dt, seed=1):
    """Rows of many scales with zeros, ties, clamped tops, subnormals, infinities and NaNs among them."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)).astype(np.float32)
    x *= np.ldexp(1.0, rng.integers(-20, 20, (rows, 1))).astype(np.float32)
    b = x.reshape(-1, 32)
    n = b.shape[0]
    special = [
        np.zeros(32), np.full(32, -0.0),
        np.r_[1.0, np.arange(31) / 128],                       # whole and half steps: ties
        np.r_[1.9921875, -1.9921875, np.full(30, 1.984375)],   # 127.5 steps and 127
        np.r_[2.0 ** -126, np.full(31, 2.0 ** -130)],          # the last normal scale
        np.r_[2.0 ** -127, np.full(31, 2.0 ** -133)],          # subnormals: scale byte 0
        np.r_[3.0e38, np.full(31, -1.0e38)], np.r_[np.inf, np.ones(31)],
        np.r_[np.ones(31), -np.inf], np.r_[np.ones(7), np.nan, np.ones(24)],
    ]
    for i, v in enumerate(special):
        b[(i * 7) % n] = v
    t = torch.from_numpy(x).to(DT[dt])
    return t, t.float().numpy()


SHAPES = [(1, 32), (1, 64), (3, 96), (77, 160), (5, 352), (130, 2048), (2, 16384), (1025, 32)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_store_and_load(dt, rows, cols):
    t, x = _values(rows, cols, dt, rows + cols)
    # the outputs sit inside larger buffers whose ends must stay as they were
    n = rows * cols
    qb = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    sb = torch.full((n // 32 + 2,), 0xAB, dtype=torch.uint8, device="cuda")
    ob = torch.full((n + 32,), 7.0, dtype=DT[dt], device="cuda")
    q, s = qb[32:32 + n].view(rows, cols), sb[1:1 + n // 32].view(rows, cols // 32)
    moe.moe_act8_store(t.cuda(), q, s)
    out = moe.moe_act8_load(q, s, DT[dt], out=ob[16:16 + n].view(rows, cols))
    torch.cuda.synchronize()
    c, e = ops.act8_encode(x)
    assert np.array_equal(to_np(s), e)
    assert np.array_equal(to_np(q).view(np.int8), c)
    ref = ops.act8_decode(c, e)
    assert np.array_equal(to_np(out).astype(np.float64), ref, equal_nan=True)
    assert (qb[:32] == 0xAB).all() and (qb[32 + n:] == 0xAB).all()
    assert sb[0] == 0xAB and sb[-1] == 0xAB
    assert (ob[:16] == 7).all() and (ob[16 + n:] == 7).all()
    # what was stored once is stored again as it is
    if not np.isnan(ref).any():
        q2, s2 = moe.moe_act8_store(out)
        assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_load_every_code_and_scale(dt):
    """All elements under all scale bytes, exact in both types."""
    c = np.arange(-127, 129).astype(np.int8)              # the last wraps to -128: left out below
    c[-1] = 0
    codes = np.tile(c, (256, 1))
    scale = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)
    q = torch.from_numpy(codes.view(np.uint8)).cuda()
    out = moe.moe_act8_load(q, torch.from_numpy(scale).cuda(), DT[dt])
    assert np.array_equal(to_np(out).astype(np.float64), ops.act8_decode(codes, scale),
                          equal_nan=True)


def test_every_bf16_value():
    """Each of the 65,536 bf16 patterns in a block of its own kind: rounded
    as the format says, beside a unit element and beside its like."""
    w = np.arange(65536, dtype=np.uint32)
    v = (w << 16).view(np.float32).reshape(-1, 1)
    half = (v.view(np.uint32) ^ 1).view(np.float32)        # its neighbour
    x = np.concatenate([v, np.ones((65536, 1), np.float32), np.zeros((65536, 30), np.float32),
                        v, half, np.zeros((65536, 30), np.float32)], axis=1)
    t = torch.from_numpy(x).bfloat16()
    q, s = moe.moe_act8_store(t.cuda())
    c, e = ops.act8_encode(t.float().numpy())
    assert np.array_equal(to_np(s), e) and np.array_equal(to_np(q).view(np.int8), c)


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    q, s = moe.moe_act8_store(e)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    assert moe.moe_act8_load(q, s).shape == (0, 64)
    ab, hp = moe.moe_act8_swiglu(q, s)
    assert ab.shape == (0, 64) and hp.shape == (0, 32)


def _near(got, ref, tol, what):
    got, ref, tol = (np.asarray(a, np.float64) for a in (got, ref, tol))
    ok = np.isnan(ref) == np.isnan(got)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - ref) <= tol) | np.isnan(ref)) | ~ok
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,h", [(1, 32), (3, 96), (130, 416), (33, 1024), (2, 8192), (4099, 64)])
def test_swiglu(dt, rows, h):
    rng = np.random.default_rng(rows + h)
    x = (rng.normal(size=(rows, 2 * h)) * np.exp(rng.normal(size=2 * h))).astype(np.float32)
    x[0, :4] = [90, -90, 30, -30]                          # a saturated gate
    if rows > 1:
        x[1, 40] = np.nan                                  # one block of NaNs
    c, e = ops.act8_encode(torch.from_numpy(x).to(DT[dt]).float().numpy())
    ref = ops.act8_decode(c, e)
    ab = torch.full((rows + 1, 2 * h), 5.0, dtype=DT[dt], device="cuda")
    hp = torch.full((rows + 1, h), 5.0, dtype=DT[dt], device="cuda")
    moe.moe_act8_swiglu(torch.from_numpy(c.view(np.uint8)).cuda(), torch.from_numpy(e).cuda(),
                        DT[dt], ab[:rows], hp[:rows])
    assert np.array_equal(to_np(ab[:rows]).astype(np.float64), ref, equal_nan=True)
    y = ops.swiglu_hidden(ref)
    tol = ((10 + 2 * np.abs(ref[:, :h])) * U + H[dt]) * np.abs(y) + 2.0 ** -126
    _near(to_np(hp[:rows]), y, tol, "hp")
    assert (ab[rows:] == 5).all() and (hp[rows:] == 5).all()


def _routing(T, E, k, seed, drop=0.0, spare=0):
    """idx, gate, token_pos (some dropped) of T tokens; R rows, `spare` of them named by nobody."""
    rng = np.random.default_rng(seed)
    lg = rng.normal(size=(T, E))
    idx = np.argsort(-lg, axis=1)[:, :k].astype(np.int32)
    g = np.exp(np.take_along_axis(lg, idx, 1))
    g = (g / g.sum(1, keepdims=True)).astype(np.float32)
    R = T * k + spare
    pos = rng.permutation(R)[:T * k].reshape(T, k).astype(np.int32)
    pos[rng.random((T, k)) < drop] = -1
    return idx, g, pos, R


COMBINE = [(1, 32, 2, 1, 0, 0), (5, 96, 8, 2, 0, 3), (37, 352, 8, 3, 0.3, 2), (64, 2080, 16, 4, 0, 0),
           (9, 256, 9, 5, 0.5, 0), (33, 544, 200, 8, 0.1, 7), (3, 16384, 4, 4, 0, 0),
           (16401, 192, 8, 1, 0.1, 1), (2050, 1056, 8, 8, 0.1, 0), (515, 8224, 5, 1, 0.2, 2)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,drop,spare", COMBINE)
def test_combine(dt, T, d, E, k, drop, spare):
    idx, g, pos, R = _routing(T, E, k, T + d, drop, spare)
    y = dev(synth.normal((R, d), 3, 0, 2.0), DT[dt])
    gd, pd = torch.from_numpy(g).cuda(), torch.from_numpy(pos).cuda()
    q = torch.full((R, d), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((R, d // 32), 0xAB, dtype=torch.uint8, device="cuda")
    out, _, _ = moe.moe_combine_act8(y, gd, pd, y8=q, y8_scale=s)
    assert torch.equal(out, moe.moe_combine(y, gd, pd))
    c, e = ops.act8_encode(to_np(y))
    named = np.zeros(R, bool)
    named[pos[pos >= 0]] = True
    assert np.array_equal(to_np(q).view(np.int8)[named], c[named])
    assert np.array_equal(to_np(s)[named], e[named])
    assert (to_np(q)[~named] == 0xAB).all() and (to_np(s)[~named] == 0xAB).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,drop,spare", COMBINE)
def test_combine_backward(dt, T, d, E, k, drop, spare):
    idx, g, pos, R = _routing(T, E, k, T + d + 1, drop, spare)
    y = to_np(dev(synth.normal((R, d), 4, 0, 2.0), DT[dt]))
    go = dev(synth.normal((T, d), 4, 1, 1.0), DT[dt])
    c, e = ops.act8_encode(y)
    v = ops.act8_decode(c, e)
    out = dict(dy_perm=torch.full((R, d), 5.0, dtype=DT[dt], device="cuda"),
               dlogits=torch.full((T, E), 5.0, device="cuda"),
               dgate=torch.full((T, k), 5.0, device="cuda"))
    args = (go, torch.from_numpy(c.view(np.uint8)).cuda(), torch.from_numpy(e).cuda(),
            torch.from_numpy(g).cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(pos).cuda(), E)
    b = moe.moe_combine_backward_act8(*args, out=out)
    ref = ops.combine_backward(to_np(go), v, g, idx, pos, E)
    named = ~np.isnan(ref["dy_perm"][:, 0])
    _near(to_np(b["dy_perm"])[named], ref["dy_perm"][named],
          (H[dt] + U) * np.abs(ref["dy_perm"][named]) + 2.0 ** -126, "dy_perm")
    assert (to_np(b["dy_perm"])[~named] == 5).all()
    mag = ops.combine_backward(np.abs(to_np(go)), np.abs(v), g, idx, pos, E)["dgate"]
    # roundings of a term: d / 64 products of a thread or fewer, d / 16 <= 16 where a token has 16
    # threads, and up to 10 additions that join them
    tol = (d / 64 + 26) * U * mag
    _near(to_np(b["dgate"]), ref["dgate"], tol + 2.0 ** -126, "dgate")
    # dlogits_i = g_i sum_j g_j (dg_i - dg_j): each dg's error, and 4k roundings of the terms
    top = g[:, :, None] * g[:, None, :]
    t2 = (top * (tol[:, :, None] + tol[:, None, :])).sum(2)
    t2 += 4 * k * U * (top * (np.abs(ref["dgate"])[:, :, None] + np.abs(ref["dgate"])[:, None, :])).sum(2)
    tl = np.zeros((T, E))
    np.put_along_axis(tl, idx.astype(np.int64), t2, 1)
    _near(to_np(b["dlogits"]), ref["dlogits"], tl + 2.0 ** -126, "dlogits")
    sel = np.zeros((T, E), bool)
    np.put_along_axis(sel, idx.astype(np.int64), True, 1)
    assert (to_np(b["dlogits"])[~sel] == 0).all()
    again = moe.moe_combine_backward_act8(*args, want_dgate=False)
    assert "dgate" not in again and torch.equal(again["dlogits"], b["dlogits"])
    assert torch.equal(again["dy_perm"][torch.from_numpy(named).cuda()],
                       b["dy_perm"][torch.from_numpy(named).cuda()])


def test_combine_backward_nan_row():
    """A row that overflowed (its checkpoint restores as NaN) reaches its own token's gradients only."""
    T, d, E, k = 6, 64, 4, 2
    idx, g, pos, R = _routing(T, E, k, 9)
    y = synth.normal((R, d), 5, 0, 1.0)
    y[pos[2, 1], 40] = np.inf
    q, s = moe.moe_act8_store(torch.from_numpy(y).cuda())
    b = moe.moe_combine_backward_act8(torch.ones(T, d, device="cuda"), q, s,
                                      torch.from_numpy(g).cuda(), torch.from_numpy(idx).cuda(),
                                      torch.from_numpy(pos).cuda(), E)
    bad = torch.isnan(b["dgate"]).cpu().numpy()
    assert bad[2, 1] and bad.sum() == 1
    assert torch.isnan(b["dlogits"]).any(1).cpu().numpy().tolist() == [False, False, True] + [False] * 3


# ---------------------------------------------------------------------------
# the layer that holds checkpoints


def _layer_in(T, d, E, k, h, seed):
    return dict(logits=synth.normal((T, E), seed, 0, 1.0), x=synth.normal((T, d), seed, 1, 1.0),
                w1=synth.normal((E, 2 * h, d), seed, 2, 0.08),
                w2=synth.normal((E, d, h), seed, 3, 0.08), dout=synth.normal((T, d), seed, 4, 1.0))


GRADS = ("dx", "dw1", "dw2", "dlogits", "dgate")


def _make(kind, inp, k, **kw):
    if kind == "mxfp8":
        return moe.MoELayerMX(dev(inp["w1"], torch.float32), dev(inp["w2"], torch.float32), k, **kw)
    return moe.MoELayer(dev(inp["w1"], DT[kind]), dev(inp["w2"], DT[kind]), k, **kw)


@pytest.mark.parametrize("kind", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("T,d,E,k,h", [(200, 256, 8, 2, 128), (1, 128, 4, 4, 128), (70, 128, 16, 3, 256)])
def test_layer(kind, T, d, E, k, h):
    """The checkpointing layer's output is the plain layer's; its gradients
    are the plain backward's on the values that its checkpoints stand for."""
    inp = _layer_in(T, d, E, k, h, 61)
    act = torch.float32 if kind == "f32" else torch.bfloat16
    x, dout, lg = dev(inp["x"], act), dev(inp["dout"], act), dev(inp["logits"], torch.float32)
    plain, layer = _make(kind, inp, k), _make(kind, inp, k, act8=True, scratch={})
    assert torch.equal(plain.forward(x, lg), layer.forward(x, lg))
    c = layer.ckpt
    for ref, q, s in ((plain.ab, "ab8", "ab8_scale"), (plain.y_perm, "y8", "y8_scale")):
        e, f = moe.moe_act8_store(ref)
        assert torch.equal(c[q], e) and torch.equal(c[s], f)
    # nothing but the checkpoints and the metadata is held: clobber the scratch
    for t in layer.scratch.values():
        t.view(torch.uint8).fill_(0xFF)
    got = {n: v.clone() for n, v in layer.backward(dout).items() if n in GRADS}
    whole = {n: v.clone() for n, v in plain.backward(dout).items() if n in GRADS}
    saved = plain.saved()
    ab, hp = moe.moe_act8_swiglu(c["ab8"], c["ab8_scale"], act)
    saved.update(ab=ab, y_perm=moe.moe_act8_load(c["y8"], c["y8_scale"], act))
    if kind != "mxfp8":
        saved["hp"] = hp
    ref = moe.moe_backward(saved, dout, E, k, d, h, mxfp8=kind == "mxfp8")
    for n in ("dx", "dw1", "dw2"):
        assert torch.equal(got[n], ref[n]), n
    # dgate is summed in another order there: d/64 + 8 roundings of its magnitudes on either side
    go = to_np(dout).astype(np.float64)
    yy = np.abs(to_np(saved["y_perm"]).astype(np.float64))[to_np(layer.route["token_pos"])]
    tol = 2 * (d / 64 + 8) * U * (np.abs(go)[:, None] * yy).sum(2)
    _near(to_np(got["dgate"]), to_np(ref["dgate"]), tol + 1e-30, "dgate")
    # and near the plain layer's: an element of a block of 32 normals is off by
    # a step / sqrt(12), the step at most its amax (about 2.1 deviations) / 64,
    # so 1 % of a deviation; dA takes a, b and dH' s', three such factors.
    # T = 1 has too few terms for a mean
    if T > 1:
        for n in ("dx", "dw1", "dw2", "dlogits"):
            assert rel_fro(to_np(got[n]), to_np(whole[n])) <= 0.03, n
    # held: A||B and y_perm at 33/32 bytes an element; x_perm and H' not at all
    # (MXFP8: H' in the layout that the plain layer holds it in as well)
    R, size = T * k, x.element_size()
    gone = R * (2 * h + d) * size + (0 if kind == "mxfp8" else R * (d + h) * size)
    assert layer.held_bytes() == plain.held_bytes() - gone + R * (2 * h + d) * 33 // 32


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
def test_layer_accumulates_and_empties(kind):
    """accumulate_dw over two micro-batches, experts without rows among them."""
    T, d, E, k, h = 96, 128, 8, 2, 128
    inp = _layer_in(T, d, E, k, h, 62)
    inp["logits"][:, 3] -= 50                              # expert 3 gets no row
    x, dout = dev(inp["x"], torch.bfloat16), dev(inp["dout"], torch.bfloat16)
    lg = dev(inp["logits"], torch.float32)
    layer = _make(kind, inp, k, act8=True, scratch={})
    layer.forward(x, lg)
    first = layer.backward(dout)["dw1"].clone()
    layer.forward(x, lg)
    twice = layer.backward(dout, accumulate_dw=True)["dw1"]
    assert torch.equal(twice, first + first)
    assert (first[3] == 0).all() and (first[0] != 0).any()


def test_layer_no_tokens():
    inp = _layer_in(1, 128, 4, 2, 128, 63)
    layer = _make("bf16", inp, 2, act8=True, scratch={})
    out = layer.forward(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"),
                        torch.empty(0, 4, device="cuda"))
    assert out.shape == (0, 128)
    g = layer.backward(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))
    assert (g["dw1"] == 0).all() and (g["dw2"] == 0).all()


@pytest.mark.parametrize("offset", [1, 4])
def test_misaligned_tensors_are_refused(offset):
    """A contiguous view that does not start on 16 bytes: an error, nothing enqueued."""
    x = torch.zeros(4 * 64 + 16, device="cuda")[offset:offset + 4 * 64].view(4, 64)
    q = torch.zeros(4 * 64 + 16, dtype=torch.uint8, device="cuda")[offset:offset + 4 * 64].view(4, 64)
    s = torch.zeros(4, 2, dtype=torch.uint8, device="cuda")
    ga = torch.ones(64, device="cuda")
    calls = [lambda: moe.moe_act8_load(q, s), lambda: moe.moe_act8_swiglu(q, s)]
    if offset % 4:
        calls += [lambda: moe.moe_act8_store(x), lambda: moe.moe_layer_norm(x, ga)]
    for call in calls:
        with pytest.raises(moe.MoeError) as err:
            call()
        assert err.value.status == moe.MOE_ERR_ALIGN
    other = torch.zeros(4, 128, device="cuda")[:, :64]
    for call in (lambda: moe.moe_act8_store(other), lambda: moe.moe_layer_norm(other, ga)):
        with pytest.raises(ValueError):
            call()                                         # rows with gaps


def test_offsets_past_32_bits():
    """More vectors than one launch takes, more bytes than 32 bits count: the
    last rows come out as they do by themselves, the rows behind stay."""
    cols = 16384
    rows = (1 << 29) // (cols // 8) + 3                    # 2^29 vectors of 8 bf16 a launch
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.fill_(0.5)
    tail = torch.randn(7, cols, device="cuda").bfloat16()
    x[-7:] = tail
    q = torch.empty((rows + 1, cols), dtype=torch.uint8, device="cuda")
    q[-1] = 9
    q, s = moe.moe_act8_store(x, q[:rows], torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda"))
    q1, s1 = moe.moe_act8_store(tail)
    assert torch.equal(q[-7:], q1) and torch.equal(s[-7:], s1) and int(q[0, 0]) == 64
    x.fill_(7)
    moe.moe_act8_load(q, s, out=x)
    assert torch.equal(x[-7:], moe.moe_act8_load(q1, s1)) and float(x[1, 1]) == 0.5
    h = cols // 2
    ab, hp = moe.moe_act8_swiglu(q, s, ab=x)
    ab1, hp1 = moe.moe_act8_swiglu(q1, s1)
    assert torch.equal(ab[-7:], ab1) and torch.equal(hp[-7:], hp1) and hp.shape == (rows, h)
