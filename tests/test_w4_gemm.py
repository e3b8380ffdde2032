"""The grouped products of MXFP8 rows with MXFP4 weights and the experts'
forward of a prompt: refusals (CPU), the kernels against 64-bit sums (GPU).

Tolerances. Where every product is a whole number of quarters, at most 16, every
partial sum of the at most 16384 products is one below 2^20: 22 bits, which fp32
holds. The one rounding is the output's: equal to the exact sum in bf16.
Otherwise the scaled
matrix instruction does not sum its products exactly in fp32 (measured 1.1e-4
of the largest sum): 1e-3 of the largest result, as for the MXFP8 GEMMs, and
the stored type's half step: bf16 2^-8 of the value; E4M3 2^-4 of the value, or
half of its smallest step, 2^-10 of the block's scale, values past 448 scales
saturated."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import oracle.w4 as w4
import routing_grouped_gemm_router_amd as moe
import synth
from helpers import dev, to_np

lib = moe.lib()
F, U = 0x100000, 0x100008
gpu = pytest.mark.gpu
U8, I32 = torch.uint8, torch.int32


def test_gemm_refusals():
    g = moe.W4GemmDesc()
    assert lib.moe_w4_gemm(None, None) == 1
    good = dict(n_groups=4, epilogue=0, rows=8, N=64, K=128, offsets=F, a_rows=None, a=F, a_scale=F, b=F,
                b_scale=F, c=F, c_scale=None)

    def status(**kw):
        for n, v in dict(good, **kw).items():
            setattr(g, n, v)
        return lib.moe_w4_gemm(ctypes.byref(g), None)

    for kw in (dict(n_groups=0), dict(n_groups=257), dict(rows=-1), dict(rows=1 << 31), dict(rows=(1 << 31) - 255), dict(N=48), dict(N=0),
               dict(N=16384 + 32), dict(K=64), dict(K=160), dict(K=16384 + 128), dict(epilogue=1, N=96, c_scale=F)):
        assert status(**kw) == 2, kw
    assert status(epilogue=2) == 3 and status(epilogue=7) == 3
    for n in ("offsets", "a", "a_scale", "b", "b_scale", "c"):
        assert status(**{n: None}) == 1, n
    assert status(c_scale=F) == 1 and status(epilogue=1) == 1
    for n in ("a", "b", "c"):
        assert status(**{n: U}) == 4, n
    for n in ("a_scale", "b_scale", "offsets", "a_rows"):
        assert status(**{n: F + 2}) == 4, n
    for n in ("a_scale", "b_scale"):
        assert status(**{n: F + 4}, K=512) == 4 and status(**{n: F + 4}, K=640, rows=0) == 0
    assert status(rows=0, a=None, c=None, offsets=None) == 0


def test_experts8_refusals():
    w = moe.W4Desc()
    good = dict(d=128, h=128, E=8, k=2, T=4, ws_bytes=1 << 20)
    for n in ("x", "topk_gate", "token_pos", "sorted_token", "offsets", "w1q", "w1_scale", "w2q",
              "w2_scale", "out", "ws"):
        good[n] = F

    def status(xs=F, **kw):
        for n, v in dict(good, **kw).items():
            setattr(w, n, v)
        return lib.moe_w4_experts8(ctypes.byref(w), xs, None)

    assert lib.moe_w4_experts8(None, F, None) == 1
    for kw in (dict(d=96), dict(d=64), dict(h=160), dict(d=16384 + 128), dict(h=8192 + 128), dict(E=0),
               dict(E=257), dict(k=0), dict(k=9, E=16), dict(k=4, E=2), dict(T=-1), dict(T=1 << 30)):
        assert status(**kw) == 2, kw
    for n in ("x", "topk_gate", "token_pos", "sorted_token", "offsets", "w1q", "w2_scale", "out", "ws"):
        assert status(**{n: None}) == 1, n
    assert status(xs=None) == 1
    for n in ("x", "out", "w1q", "w2q", "ws"):
        assert status(**{n: U}) == 4, n
    assert status(w1_scale=F + 2) == 4 and status(w2_scale=F + 1) == 4 and status(xs=F + 2) == 4
    assert status(d=512, w1_scale=F + 4) == 4 and status(d=512, xs=F + 4) == 4 and status(h=512, w2_scale=F + 4) == 4
    need = moe.moe_w4_experts8_workspace_size(4, 2, 128, 128)
    assert need == 8 * 128 + 256 + 8 * 128 * 2 + 256 and status(ws_bytes=need - 1) == 5
    assert status(T=0, x=None, out=None, ws=None) == 0
    assert moe.moe_w4_experts8_workspace_size(4, 2, 96, 128) == 0


def test_binding_refusals():
    z = lambda *s: torch.zeros(*s, dtype=U8)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w4_gemm(z(4, 128), z(4, 4), z(2, 64, 64), z(2, 64, 4), torch.zeros(3, dtype=I32))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w4_experts8(z(4, 128), z(4, 4), {}, z(2, 256, 64), z(2, 256, 4), z(2, 128, 64), z(2, 128, 4))


# ---------------------------------------------------------------------------


def _whole(shape, rng, fill):
    """Whole numbers -2 .. 2, most of them zero, under scales of 1/2, 1 or 2."""
    v = rng.integers(-2, 3, shape) * (rng.random(shape) < fill)
    s = rng.integers(126, 129, shape[:-1] + (shape[-1] // 32,))
    return v.astype(np.float64), s.astype(np.uint8)


def _e4m3(v):
    """E4M3 bytes of whole numbers -2 .. 2."""
    return (np.array([0, 0x38, 0x40], np.uint8)[np.abs(v).astype(int)] | (np.signbit(v) * 0x80).astype(np.uint8))


def _e2m1(v):
    return w4.pack(np.array([0, 2, 4], np.uint8)[np.abs(v).astype(int)] | (np.signbit(v) * 8).astype(np.uint8))


def _val(v, s):
    return v * np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=-1)


def _cuda(*a):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in a]


def _groups(kind, E, rng):
    if kind == "edges":                           # around the tiles' ends, empty ones among them
        return [0, 1, 127, 128, 129, 0, 31, 32, 33, 63, 64, 65, 255, 257, 0, 2][:E] + [5] * max(0, E - 16)
    if kind == "one":
        return [0] * (E - 1) + [300]
    return list(rng.integers(0, 40, E))


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kind,E,N,K", [
    ("edges", 16, 32, 128), ("edges", 16, 256, 256), ("edges", 16, 288, 384), ("one", 1, 64, 128),
    ("one", 3, 544, 640), ("few", 256, 96, 128), ("few", 40, 1056, 128), ("few", 5, 128, 16384),
    ("one", 2, 16384, 128), ("edges", 7, 416, 640)])
def test_whole_numbers(kind, E, N, K, gather):
    """Sums that fp32 holds: every output equal, rows outside all groups and
    around the output left as they were."""
    rng = np.random.default_rng(E * N + K + gather)
    counts = _groups(kind, E, rng)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1])
    total = R // 3 + 7 if gather else R + 9       # a's rows
    a, sa = _whole((total, K), rng, min(1.0, 24 / K))
    b, sb = _whole((E, N, K), rng, 0.5)
    rows = rng.integers(0, total, R + 9).astype(np.int32) if gather else np.arange(R + 9, dtype=np.int32)
    av, bv = _val(a, sa), _val(b, sb)
    out = torch.full((R + 9 + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    aq, as_, bq, bs, o, ar = _cuda(_e4m3(a), sa, _e2m1(b), sb, off, rows)
    got = moe.moe_w4_gemm(aq, as_, bq, bs, o, a_rows=ar if gather else None, out=out[1:-1])
    ref = np.zeros((R, N))
    for e in range(E):
        r = rows[off[e]:off[e + 1]]
        ref[off[e]:off[e + 1]] = av[r] @ bv[e].T
    want = torch.from_numpy(ref).to(torch.bfloat16)
    assert np.array_equal(ref * 4, np.rint(ref * 4))
    assert torch.equal(got[:R].cpu(), want)
    assert (out[0] == 7).all() and (out[R + 1:] == 7).all()


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("E,N,K,counts", [
    (3, 16384, 128, (300, 0, 213)), (8, 8192, 384, (130, 64, 256, 0, 1, 127, 129, 400)),
    (2, 16384, 512, (385, 640)), (5, 2080, 640, (700, 13, 129, 500, 255)),
    (2, 4096, 512, (150, 61)), (6, 1056, 1024, (90, 190, 33, 0, 64, 65)),
    # medium tiles
    (2, 8192, 512, (300, 261)), (6, 4128, 1024, (190, 250, 133, 0, 64, 65)), (1, 16384, 640, (250,)),
    # large ones, with scales of one step and of four at a time
    (3, 16384, 640, (700, 33, 500)), (4, 16384, 1024, (700, 33, 500, 129))])
def test_whole_numbers_many_rows(E, N, K, counts, gather):
    """The larger tiles' sizes, on sums that fp32 holds; every group by itself
    (small tiles) gives the same bits on values that are rounded."""
    rng = np.random.default_rng(N + K + gather)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1])
    total = R // 2 if gather else R
    a, sa = _whole((total, K), rng, min(1.0, 24 / K))
    b, sb = _whole((E, N, K), rng, 0.5)
    rows = rng.integers(0, total, R).astype(np.int32) if gather else np.arange(R, dtype=np.int32)
    aq, as_, bq, bs, o, ar = _cuda(_e4m3(a), sa, _e2m1(b), sb, off, rows)
    got = moe.moe_w4_gemm(aq, as_, bq, bs, o, a_rows=ar if gather else None)
    av, bv = _val(a, sa), _val(b, sb)
    ref = np.concatenate([av[rows[off[e]:off[e + 1]]] @ bv[e].T for e in range(E)])
    assert torch.equal(got.cpu(), torch.from_numpy(ref).to(torch.bfloat16))
    x = torch.randint(0, 256, aq.shape, dtype=U8, device="cuda")
    x[(x & 0x7F) == 0x7F] = 0x70                            # no NaNs
    w = torch.randint(0, 256, bq.shape, dtype=U8, device="cuda")
    epi = moe.MOE_EPI_SWIGLU_FWD if N % 64 == 0 else moe.MOE_EPI_NONE
    for ep in {moe.MOE_EPI_NONE, epi}:
        whole = moe.moe_w4_gemm(x, as_, w, bs, o, ep, ar if gather else None)
        for e in range(E):
            sl = slice(int(off[e]), min(int(off[e + 1]), int(off[e]) + 40))
            if sl.start == sl.stop:
                continue
            one = moe.moe_w4_gemm(x, as_, w[e:e + 1], bs[e:e + 1],
                                  torch.tensor([0, sl.stop - sl.start], dtype=I32, device="cuda"), ep,
                                  ar[sl].contiguous() if gather else torch.arange(sl.start, sl.stop, dtype=I32,
                                                                                  device="cuda"))
            for p, q in zip(whole if ep else (whole,), one if ep else (one,)):
                assert torch.equal(p[sl], q), (ep, e)


def _real(rows, cols, seed, i):
    x = synth.normal((rows, cols), seed, i, 1.0) * np.exp(0.5 * synth.normal((1, cols), seed, i + 50, 1.0))
    q, s = oracle.mxfp8_quantize(x.astype(np.float32), 1)
    q, s = np.asarray(q).reshape(rows, cols), np.asarray(s).reshape(rows, cols // 32)
    return q, s, np.asarray(oracle.mxfp8_dequantize_rowwise(q, s), np.float64)


def _real4(E, rows, cols, seed, i):
    c, s = w4.encode(synth.normal((E * rows, cols), seed, i, cols ** -0.5))
    v = w4.decode(c, s).reshape(E, rows, cols)
    return w4.pack(c).reshape(E, rows, cols // 2), s.reshape(E, rows, cols // 32), v


@gpu
@pytest.mark.parametrize("T,K,N,E,k", [(1, 128, 128, 2, 1), (200, 512, 544, 5, 2), (333, 2048, 256, 8, 4),
                                       (64, 1024, 2048, 64, 8)])
def test_values(T, K, N, E, k):
    rng = np.random.default_rng(T)
    q, s, v = _real(T, K, 61, 0)
    bq, bs, bv = _real4(E, N, K, 61, 1)
    r = moe.moe_route(dev(rng.normal(size=(T, E)), torch.float32), k)
    aq, as_, bq, bs = _cuda(q, s, bq, bs)
    got = to_np(moe.moe_w4_gemm(aq, as_, bq, bs, r["offsets"], a_rows=r["sorted_token"]))
    off, tok = to_np(r["offsets"]), to_np(r["sorted_token"])
    ref = np.concatenate([v[tok[off[e]:off[e + 1]]] @ bv[e].T for e in range(E)])
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-3 * np.abs(ref).max()).all()
    perm = moe.moe_permute(aq, r["token_pos"], x_scale=as_)
    assert np.array_equal(to_np(moe.moe_w4_gemm(perm[0], perm[1], bq, bs, r["offsets"])), got)


def _silu(a):
    e = np.exp(-np.abs(a))
    return np.where(a < 0, a * e, a) / (1 + e)


@gpu
@pytest.mark.parametrize("T,d,h,E,k", [(1, 128, 32, 2, 1), (130, 256, 96, 3, 1), (300, 512, 160, 5, 2),
                                       (77, 1024, 1024, 4, 4)])
def test_swiglu(T, d, h, E, k):
    """H' in MXFP8: the scale of its block's largest value (one off only where
    that lies within the product's error of a power of two), each element
    within half a step."""
    q, s, v = _real(T, d, 62, 0)
    bq, bs, bv = _real4(E, 2 * h, d, 62, 1)
    r = moe.moe_route(dev(synth.normal((T, E), 62, 2, 1.0), torch.float32), k)
    R = T * k
    aq, as_, bq, bs = _cuda(q, s, bq, bs)
    big = torch.full((R * h + 32,), 0xAB, dtype=U8, device="cuda")
    bigs = torch.full((R * h // 32 + 8,), 0xAB, dtype=U8, device="cuda")
    hq, hs = big[16:16 + R * h].view(R, h), bigs[4:4 + R * h // 32].view(R, h // 32)
    moe.moe_w4_gemm(aq, as_, bq, bs, r["offsets"], moe.MOE_EPI_SWIGLU_FWD, r["sorted_token"], hq, hs)
    assert (big[:16] == 0xAB).all() and (big[-16:] == 0xAB).all()
    assert (bigs[:4] == 0xAB).all() and (bigs[-4:] == 0xAB).all()
    off, tok = to_np(r["offsets"]), to_np(r["sorted_token"])
    ab = np.concatenate([v[tok[off[e]:off[e + 1]]] @ bv[e].T for e in range(E)])
    a, b = ab[:, :h], ab[:, h:]
    ref = _silu(a) * b
    err = 1e-3 * np.abs(ab).max()
    eh = (err * (1.1 * np.abs(b) + np.abs(_silu(a)) + err) + 1e-5 * np.abs(ref))
    scale = to_np(hs).astype(int)
    amax, ea = np.abs(ref).reshape(R, -1, 32).max(2), eh.reshape(R, -1, 32).max(2)
    exp = lambda x: np.maximum(np.frexp(x)[1] - 1 + 127 - 8, 0)
    assert ((scale >= exp(np.maximum(amax - ea, 1e-30))) & (scale <= exp(amax + ea))).all()
    step = np.repeat(np.ldexp(1.0, scale - 127), 32, axis=1)
    got = np.asarray(oracle.mxfp8_dequantize_rowwise(to_np(hq), to_np(hs)), np.float64)
    want = np.clip(ref, -448 * step, 448 * step)
    assert (np.abs(got - want) <= eh * (1 + 2.0 ** -3) + 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * step).all()


def _layer(T, d, h, E, k, seed):
    q, s, v = _real(T, d, seed, 0)
    w1, w2 = _real4(E, 2 * h, d, seed, 1), _real4(E, d, h, seed, 2)
    r = moe.moe_route(dev(synth.normal((T, E), seed, 3, 1.0), torch.float32), k)
    return _cuda(q, s), v, w1, w2, _cuda(w1[0], w1[1], w2[0], w2[1]), r


@gpu
@pytest.mark.parametrize("T,d,h,E,k", [(1, 128, 128, 2, 1), (5, 256, 128, 256, 8), (150, 512, 256, 5, 2),
                                       (1030, 384, 640, 8, 3), (600, 2048, 1024, 16, 4), (40, 2432, 128, 4, 2),
                                       (9, 16384, 128, 2, 2)])
def test_experts8(T, d, h, E, k):
    """The calls that it is made of, to their roundings; the whole against 64 bits.

    Its tolerance by arithmetic: with X = 2^(floor(log2 amax) - 8), a block's
    scale, an element of H' is off by at most 2^-4 of itself or 2^-10 X, X <=
    2^-8 amax; one above 448 X is taken to 448 X, by less than 64 X, an eighth of
    itself. The down product carries the sum of these magnitudes, 2^-3 |H'| +
    2^-18 amax, into an output. The products' own errors are 1e-3 of their
    largest result (see above), a and b's through H' by silu' <= 1.1; then y is
    rounded to fp16 with its block's largest between 2^14 and 2^15, 2^-11 of the
    value or half of a smallest step, 2^-25 in 2^14 of the largest, and out to
    bf16, 2^-8."""
    (xq, xs), v, w1, w2, w, r = _layer(T, d, h, E, k, 63)
    got = moe.moe_w4_experts8(xq, xs, r, *w)
    hq, hs = moe.moe_w4_gemm(xq, xs, w[0], w[1], r["offsets"], moe.MOE_EPI_SWIGLU_FWD, r["sorted_token"])
    y = moe.moe_w4_gemm(hq, hs, w[2], w[3], r["offsets"])
    idx, gate = to_np(r["topk_idx"]), to_np(r["topk_gate"])
    # the sum of y in bf16 (2^-8 of each term and of the result), fp32's own errors
    # beside it nothing
    parts = np.abs(to_np(y)[to_np(r["token_pos"])].astype(np.float64)) * gate[:, :, None]
    whole = to_np(moe.moe_combine(y, r["topk_gate"], r["token_pos"])).astype(np.float64)
    assert (np.abs(to_np(got) - whole) <= (2.0 ** -8 + 2.0 ** -10) * parts.sum(1) + 2.0 ** -7 * np.abs(whole)).all()
    ref, tol = np.zeros((T, d)), np.zeros((T, d))
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if len(t):
            ab = v[t] @ w1[2][e].T
            a, b = ab[:, :h], ab[:, h:]
            hid = _silu(a) * b
            err = 1e-3 * np.abs(ab).max()
            eh = err * (1.1 * np.abs(b) + np.abs(_silu(a)) + 1.1 * err)
            amax = np.repeat(np.abs(hid).reshape(len(t), -1, 32).max(2), 32, axis=1)
            eh = eh * (1 + 2.0 ** -3) + 2.0 ** -3 * np.abs(hid) + 2.0 ** -18 * amax
            out, ey = hid @ w2[2][e].T, eh @ np.abs(w2[2][e]).T
            ey = ey + 1e-3 * np.abs(out).max()
            most = np.repeat((np.abs(out) + ey).reshape(len(t), -1, 32).max(2), 32, axis=1)
            ey = ey + 2.0 ** -11 * (np.abs(out) + ey) + 2.0 ** -39 * most
            ref[t] += gate[t, j][:, None] * out
            tol[t] += gate[t, j][:, None] * ey
    assert (np.abs(to_np(got) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()


@gpu
def test_experts8_of_many_magnitudes():
    """Outputs of one token from 2^-70 to 2^70, next to each other and block by
    block: each as near as its own magnitude lets fp16 of the block's scale be. H' =
    silu(a) b is a whole block of the same value, which E4M3 holds, so that y's is
    the only rounding but out's."""
    T, d, h, E = 70, 512, 128, 3
    one = lambda *s: torch.full(s, 127, dtype=U8, device="cuda")
    xq = torch.full((T, d), 0x38, dtype=U8, device="cuda")              # ones
    w1 = torch.zeros(E, 2 * h, d // 2, dtype=U8, device="cuda")
    w1[:, :h, 0] = 0x07                                                 # a = 6
    w1[:, h:, 0] = 0x02                                                 # b = 1
    rng = np.random.default_rng(5)
    c = rng.integers(0, 16, (E, d, h)).astype(np.uint8)
    base = np.repeat(rng.integers(60, 190, (E, d // 32)), 32, axis=1)
    s2 = np.repeat((base + rng.integers(-8, 9, (E, d)))[:, :, None], h // 32, axis=2).astype(np.uint8)
    w2, s2c = _cuda(w4.pack(c.reshape(E * d, h)).reshape(E, d, h // 2), s2)
    r = moe.moe_route(dev(synth.normal((T, E), 70, 0, 1.0), torch.float32), 1)
    got = to_np(moe.moe_w4_experts8(xq, one(T, d // 32), r, w1, one(E, 2 * h, d // 32), w2, s2c)).astype(np.float64)
    hq, hs = moe.moe_w4_gemm(xq, one(T, d // 32), w1, one(E, 2 * h, d // 32), r["offsets"], moe.MOE_EPI_SWIGLU_FWD,
                             r["sorted_token"])
    hid = float(oracle.mxfp8_dequantize_rowwise(to_np(hq), to_np(hs))[0, 0])
    y = hid * w4.decode(c.reshape(E * d, h), s2.reshape(E * d, h // 32)).reshape(E, d, h).sum(2)
    ref = y[to_np(r["topk_idx"])[:, 0]]
    top = hid * np.abs(w4.decode(c.reshape(E * d, h), s2.reshape(E * d, h // 32))).reshape(E, d, h).sum(2)
    err = 1e-4 * top                                                    # the matrix units' sums
    most = np.repeat((np.abs(y) + err).reshape(E, -1, 32).max(2), 32, axis=1)
    tol = (err + 2.0 ** -11 * (np.abs(y) + err) + 2.0 ** -39 * most)[to_np(r["topk_idx"])[:, 0]]
    assert np.isfinite(got).all() and np.abs(ref).max() > 2.0 ** 50 and np.abs(ref[ref != 0]).min() < 2.0 ** -50
    assert (np.abs(got - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()


@gpu
def test_skewed_experts():
    """One expert with most rows, many with none."""
    T, d, h, E, k = 900, 256, 128, 40, 2
    q, s, v = _real(T, d, 64, 0)
    w1, w2 = _real4(E, 2 * h, d, 64, 1), _real4(E, d, h, 64, 2)
    logits = synth.normal((T, E), 64, 3, 0.1)
    logits[:, 17] += 10
    logits[:, 20:] -= 20
    r = moe.moe_route(dev(logits, torch.float32), k)
    aq, as_, b1, s1 = _cuda(q, s, w1[0], w1[1])
    got = to_np(moe.moe_w4_gemm(aq, as_, b1, s1, r["offsets"], a_rows=r["sorted_token"]))
    off, tok = to_np(r["offsets"]), to_np(r["sorted_token"])
    assert off[18] - off[17] == T and off[40] == off[20]
    ref = np.concatenate([v[tok[off[e]:off[e + 1]]] @ w1[2][e].T for e in range(E)])
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-3 * np.abs(ref).max()).all()


@gpu
def test_nan_rows_stay_alone():
    """A token whose scales and elements are NaN, in a group with others."""
    (xq, xs), v, w1, w2, w, r = _layer(100, 256, 128, 2, 1, 65)
    clean = moe.moe_w4_experts8(xq, xs, r, *w)
    xq, xs = xq.clone(), xs.clone()
    xq[7] = 0x7F
    xs[41] = 255
    out = moe.moe_w4_experts8(xq, xs, r, *w)
    keep = [i for i in range(100) if i not in (7, 41)]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[7]).all() and torch.isnan(out[41]).all()


@gpu
def test_rows_past_32_bits():
    """Gathered rows whose byte offsets pass 2^32."""
    K, N, rows = 8192, 64, (1 << 19) + 40
    a = torch.zeros(rows, K, dtype=U8, device="cuda")
    s = torch.full((rows, K // 32), 127, dtype=U8, device="cuda")
    a[-1, :4], a[5, 100] = 0x38, 0x40                        # ones; a two
    b = torch.full((1, N, K // 2), 0x22, dtype=U8, device="cuda")     # ones
    bs = torch.full((1, N, K // 32), 127, dtype=U8, device="cuda")
    off = torch.tensor([0, 3], dtype=I32, device="cuda")
    at = torch.tensor([rows - 1, 5, rows - 2], dtype=I32, device="cuda")
    got = moe.moe_w4_gemm(a, s, b, bs, off, a_rows=at)
    assert (got[0] == 4).all() and (got[1] == 2).all() and (got[2] == 0).all()


@gpu
def test_prompt_object():
    """MoELayerW4.prompt on bf16 rows and on the norm's 8-bit rows, in turn with
    the few-token forward; replays of a captured prompt on new logits."""
    T, d, h, E, k = 200, 256, 128, 8, 2
    n = lambda sh, i, c=1.0: synth.normal(sh, 66, i, c)
    w1, w2 = dev(n((E, 2 * h, d), 0, d ** -0.5), torch.float32), dev(n((E, d, h), 1, h ** -0.5), torch.float32)
    x, res = dev(n((T, d), 2), torch.bfloat16), dev(n((T, d), 3), torch.bfloat16)
    wr = dev(n((E, d), 4, d ** -0.5), torch.float32)
    layer = moe.MoELayerW4(w1, w2, k)
    norm = moe.RMSNorm(dev(1 + n((d,), 5, 0.1), torch.float32), quantize=True)
    y = norm.forward(x, res)
    logits = y.float() @ wr.t()
    a = layer.prompt(y, logits).clone()
    r = moe.moe_route(logits, k)
    assert torch.equal(a, moe.moe_w4_experts8(*norm.q, r, layer.w1q, layer.w1s, layer.w2q, layer.w2s))
    few = layer.forward(y[:3].contiguous(), logits[:3].contiguous()).clone()
    assert torch.equal(a, layer.prompt(None, logits, xq=norm.q))
    assert torch.equal(few, layer.forward(y[:3].contiguous(), logits[:3].contiguous()))
    graph = torch.cuda.CUDAGraph()
    layer.prompt(y, logits)
    with torch.cuda.graph(graph):
        norm.forward(x, res)
        out = layer.prompt(None, logits, xq=norm.q)
    for i in range(3):
        logits.copy_(dev(n((T, E), 10 + i), torch.float32))
        x.copy_(dev(n((T, d), 20 + i), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        f = moe.moe_rms_norm(x, norm.weight, norm.eps, res, quantize=True, want_y=False, stats=False)
        want = moe.moe_w4_experts8(f["yq"], f["yq_scale"], moe.moe_route(logits, k), layer.w1q, layer.w1s,
                                   layer.w2q, layer.w2s)
        assert torch.equal(out, want), i
    with pytest.raises(ValueError, match="x is required|x: expected"):
        layer.prompt(None, logits)
    with pytest.raises(ValueError, match="xq"):
        layer.prompt(None, logits, xq=(norm.q[0][:5], norm.q[1][:5]))


@gpu
def test_another_stream():
    """On a stream of its own, behind work that makes the inputs there."""
    (xq, xs), v, w1, w2, w, r = _layer(300, 256, 128, 4, 2, 67)
    want = moe.moe_w4_experts8(xq, xs, r, *w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2, s2 = torch.zeros_like(xq), torch.zeros_like(xs)
        x2.copy_(xq)
        s2.copy_(xs)
        got = moe.moe_w4_experts8(x2, s2, r, *w)
    side.synchronize()
    assert torch.equal(got, want)


@gpu
def test_dropped_slots():
    """Slots with a negative position add nothing; their rows are computed."""
    (xq, xs), v, w1, w2, w, r = _layer(50, 128, 128, 3, 2, 68)
    full = moe.moe_w4_experts8(xq, xs, r, *w)
    cut = dict(r, token_pos=r["token_pos"].clone(), topk_gate=r["topk_gate"].clone())
    cut["token_pos"][::3, 1] = -1
    got = moe.moe_w4_experts8(xq, xs, cut, *w)
    gate = r["topk_gate"].clone()
    gate[::3, 1] = 0
    want = moe.moe_w4_experts8(xq, xs, dict(r, topk_gate=gate), *w)
    assert torch.equal(got, want) and not torch.equal(got, full)


@gpu
def test_no_rows_and_refusals():
    d, h, E = 128, 128, 4
    z = lambda *s: torch.zeros(*s, dtype=U8, device="cuda")
    w = (z(E, 2 * h, d // 2), z(E, 2 * h, d // 32), z(E, d, h // 2), z(E, d, h // 32))
    off = torch.zeros(E + 1, dtype=I32, device="cuda")
    assert moe.moe_w4_gemm(z(0, d), z(0, 4), w[0], w[1], off).shape == (0, 2 * h)
    out = torch.full((3, 2 * h), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_gemm(z(3, d), z(3, 4), w[0], w[1], off, out=out)          # every group empty
    assert (out == 5).all()
    r = moe.moe_route(torch.zeros(0, E, device="cuda"), 2)
    assert moe.moe_w4_experts8(z(0, d), z(0, 4), r, *w).shape == (0, d)
    with pytest.raises(ValueError, match="out_scale"):
        moe.moe_w4_gemm(z(3, d), z(3, 4), w[0], w[1], off, out_scale=z(3, 4))
    with pytest.raises(ValueError, match="b_scale"):
        moe.moe_w4_gemm(z(3, d), z(3, 4), w[0], w[1][:1], off)
    with pytest.raises(ValueError, match="offsets"):
        moe.moe_w4_gemm(z(3, d), z(3, 4), w[0], w[1], off[:3])
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_w4_gemm(z(3, 64), z(3, 2), z(E, 64, 32), z(E, 64, 2), off)
    r = moe.moe_route(torch.zeros(3, E, device="cuda"), 2)
    with pytest.raises(ValueError, match="ws"):
        moe.moe_w4_experts8(z(3, d), z(3, 4), r, *w, ws=z(16))


# T, d, h, E, k of experts whose down product takes each tile with scales of one step
# (h no multiple of 512) and of four; on the larger tiles also a d that leaves some
# of the last tile's columns past its end.
FORMS = [(1000, 640, 128, 32, 1), (1000, 512, 512, 32, 1), (3, 4224, 1024, 2, 1),            # small
         (600, 8064, 640, 2, 1), (600, 8192, 512, 2, 1),                                     # medium
         (1400, 16384, 128, 2, 1), (1400, 16256, 640, 2, 1), (1400, 16384, 512, 2, 1),       # large
         (1400, 16256, 1024, 2, 1)]


@gpu
@pytest.mark.parametrize("T,d,h,E,k", FORMS)
def test_experts8_exact_on_every_tile(T, d, h, E, k):
    """H' known and held by E4M3, y a whole number of half-units that fp32's sums and
    fp16 of a block's scale hold: out is y rounded once.

    Gate inputs are 6, whose silu, 5.985, goes to 6 under any power of two; the up
    inputs b = x[t, c] u[j] are 0 or up to 4 in magnitude, so H' = 6 b. y / 6 = sum_j
    b_j w2[n, j] is a whole number of halves, at most 341 (asserted): y has 11 bits."""
    rng = np.random.default_rng(d + h)
    xv = np.zeros((T, d))
    xv[:, 0] = 1
    xv[:, 1:5] = rng.integers(-2, 3, (T, 4))
    u, col = rng.integers(-2, 3, (E, h)), rng.integers(1, 5, (E, h))
    w1 = np.zeros((E, 2 * h, d), np.int8)
    w1[np.arange(E)[:, None], h + np.arange(h), col] = u
    code = np.array([4 | 8, 2 | 8, 0, 2, 4], np.uint8)[w1 + 2]        # -2 .. 2 in E2M1
    code[:, :h, 0] = 7                                                # 6
    c, sc = _whole((E, d, h), rng, min(1.0, 16 / h))
    w2 = _val(c, sc)
    part = np.stack([np.where(col == i, u, 0) for i in range(1, 5)], 1).astype(np.float64)     # [E, 4, h]
    v = np.stack([w2[e] @ part[e].T for e in range(E)])               # [E, d, 4]
    r = moe.moe_route(dev(rng.normal(size=(T, E)), torch.float32), k)
    idx = to_np(r["topk_idx"])[:, 0]
    ref = np.zeros((T, d))
    for e in range(E):
        ref[idx == e] = xv[idx == e, 1:5] @ v[e].T
    assert np.abs(ref).max() <= 341 and np.array_equal(2 * ref, np.rint(2 * ref)) and (to_np(r["topk_gate"]) == 1).all()
    one = lambda *s: torch.full(s, 127, dtype=U8, device="cuda")
    xq, w1q, w2q, w2s = _cuda(_e4m3(xv), w4.pack(code.reshape(E * 2 * h, d)).reshape(E, 2 * h, d // 2), _e2m1(c), sc)
    got = moe.moe_w4_experts8(xq, one(T, d // 32), r, w1q, one(E, 2 * h, d // 32), w2q, w2s)
    assert torch.equal(got.cpu(), torch.from_numpy(6 * ref).to(torch.bfloat16))


def _random_experts(T, d, h, E, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = [t.view(E, -1, t.shape[-1]) for rows, cols in ((2 * h, d), (d, h))
         for t in moe.moe_w4_quantize(n(E * rows, cols) * cols ** -0.5)]
    return moe.mxfp8_quantize(n(T, d), 1), w, n(T, E)


@gpu
@pytest.mark.parametrize("T,d,h,E,k", [(T // 2 if E == 2 and T > 3 else T, d, h, E, 2) for T, d, h, E, _ in FORMS] +
                         [(100, 4224, 128, 16, 8), (90, 2176, 512, 16, 5), (33, 7168, 256, 8, 7)])
def test_experts8_tokens_by_themselves(T, d, h, E, k):
    """A token's result does not depend on the others, whatever tile their number
    leads to, nor on the call: the first 40 by themselves give the same bits."""
    (xq, xs), w, logits = _random_experts(T, d, h, E, k, T + d)
    full = moe.moe_w4_experts8(xq, xs, moe.moe_route(logits, k), *w)
    assert torch.equal(full, moe.moe_w4_experts8(xq, xs, moe.moe_route(logits, k), *w))
    n = min(T, 40)
    few = moe.moe_w4_experts8(xq[:n], xs[:n], moe.moe_route(logits[:n].contiguous(), k), *w)
    assert torch.isfinite(full).all() and full.abs().max() > 0.5
    assert torch.equal(full[:n], few)


@gpu
@pytest.mark.parametrize("T,d,h,E,k", [(100, 4224, 128, 16, 8), (33, 2176, 256, 8, 6)])
def test_experts8_of_many_slots(T, d, h, E, k):
    """Five to eight slots a token with rows of more than one piece of the combine."""
    test_experts8(T, d, h, E, k)


@gpu
def test_experts8_of_many_tokens():
    """2^26 tokens and more, of which one launch of the combine takes 2^23: every
    1024 of them the same, and the same as 1024 by themselves."""
    T, n, d, h = (1 << 26) + 1024 + 5, 1024, 128, 128
    (xq, xs), w, _ = _random_experts(n, d, h, 1, 1, 9)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    gate = torch.rand((n, 1), generator=g, device="cuda")
    over = lambda t: t.repeat((T + n - 1) // n, 1)[:T]
    pos = torch.arange(T, dtype=I32, device="cuda")
    route = lambda m, gt: dict(topk_gate=gt, token_pos=pos[:m, None], sorted_token=pos[:m],
                               offsets=torch.tensor([0, m], dtype=I32, device="cuda"))
    want = moe.moe_w4_experts8(xq, xs, route(n, gate), *w)
    out = torch.full((T + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_experts8(over(xq), over(xs), route(T, over(gate)), *w, out=out[:T])
    assert (out[T] == 7).all() and torch.equal(out[T // n * n:T], want[:T % n])
    for part in out[:T // n * n].view(-1, n, d).split(4096):
        assert (part == want).all()


def test_experts8_rows_past_the_products():
    """The products' rows end at 2^31 - 256; so do the experts' T k."""
    w = moe.W4Desc()
    for n, v in dict(d=128, h=128, E=8, ws_bytes=1 << 62).items():
        setattr(w, n, v)
    for n in ("x", "topk_gate", "token_pos", "sorted_token", "offsets", "w1q", "w1_scale", "w2q", "w2_scale", "out"):
        setattr(w, n, F)
    size = moe.moe_w4_experts8_workspace_size
    for T, k in (((1 << 31) - 255, 1), ((1 << 30) - 127, 2), ((1 << 28) - 31, 8)):
        w.T, w.k, w.ws = T, k, F
        assert lib.moe_w4_experts8(ctypes.byref(w), F, None) == 2 and size(T, k, 128, 128) == 0
        w.T, w.ws = T - 1, None                       # the last one of a size: the next check's turn
        assert lib.moe_w4_experts8(ctypes.byref(w), F, None) == 1 and size(T - 1, k, 128, 128) > 0
