"""Refusals of the 8-bit checkpoint and layer norm calls (no GPU needed): each
bad argument gives the documented status before anything is enqueued, and the
binding raises on tensors that do not fit."""
import ctypes

import pytest
import torch

import routing_grouped_gemm_router_amd as moe

F = 0x100000          # never dereferenced: validation fails first
U = F + 4             # not 16-byte aligned
NULL, SHAPE, DTYPE, ALIGN, WS = 1, 2, 3, 4, 5
BF16, F32 = moe.MOE_BF16, moe.MOE_F32
lib = moe.lib()


@pytest.mark.parametrize("args,st", [
    ((F, moe.MOE_MXFP8, 4, 64, F, F, None), DTYPE),
    ((F, 7, 4, 64, F, F, None), DTYPE),
    ((F, BF16, -1, 64, F, F, None), SHAPE),
    ((F, BF16, 1 << 31, 64, F, F, None), SHAPE),
    ((F, BF16, 4, 48, F, F, None), SHAPE),
    ((F, BF16, 4, 0, F, F, None), SHAPE),
    ((F, BF16, 4, 1 << 20, F, F, None), SHAPE),
    ((None, BF16, 4, 64, F, F, None), NULL),
    ((F, BF16, 4, 64, None, F, None), NULL),
    ((F, BF16, 4, 64, F, None, None), NULL),
    ((U, BF16, 4, 64, F, F, None), ALIGN),
    ((F, BF16, 4, 64, U, F, None), ALIGN),
    ((None, BF16, 0, 64, None, None, None), 0),
])
def test_act8_store(args, st):
    assert lib.moe_act8_store(*args) == st


@pytest.mark.parametrize("args,st", [
    ((F, F, moe.MOE_MXFP8, 4, 64, F, None), DTYPE),
    ((F, F, F32, 4, 33, F, None), SHAPE),
    ((None, F, F32, 4, 64, F, None), NULL),
    ((F, None, F32, 4, 64, F, None), NULL),
    ((F, F, F32, 4, 64, None, None), NULL),
    ((F, F, F32, 4, 64, U, None), ALIGN),
    ((U, F, F32, 4, 64, F, None), ALIGN),
    ((None, None, F32, 0, 64, None, None), 0),
])
def test_act8_load(args, st):
    assert lib.moe_act8_load(*args) == st


@pytest.mark.parametrize("args,st", [
    ((F, F, moe.MOE_MXFP8, 4, 64, F, F, None), DTYPE),
    ((F, F, BF16, 4, 48, F, F, None), SHAPE),
    ((F, F, BF16, 4, 8192 + 32, F, F, None), SHAPE),       # 2h <= 16384
    ((F, F, BF16, -4, 64, F, F, None), SHAPE),
    ((F, F, BF16, 4, 64, None, F, None), NULL),
    ((F, F, BF16, 4, 64, F, None, None), NULL),
    ((F, F, BF16, 4, 64, F, U, None), ALIGN),
    ((None, None, BF16, 0, 64, None, None, None), 0),
])
def test_act8_swiglu(args, st):
    assert lib.moe_act8_swiglu(*args) == st


def combine(dt=BF16, T=16, d=64, k=2, y=F, out=F, y8=F, sc=F):
    return lib.moe_combine_act8(y, dt, F, F, T, d, k, out, y8, sc, None)


def combine_bwd(dt=BF16, T=16, d=64, k=2, E=8, dout=F, y8=F, sc=F, dy=F, dl=F):
    return lib.moe_combine_backward_act8(dout, dt, y8, sc, F, F, F, T, d, k, E, dy, dl, None, None)


def test_combine_act8():
    assert combine(dt=2) == DTYPE
    assert combine(T=-1) == SHAPE and combine(d=48) == SHAPE and combine(d=16384 + 32) == SHAPE
    assert combine(k=0) == SHAPE and combine(k=9) == SHAPE and combine(T=1 << 30, k=4) == SHAPE
    assert combine(y=None) == NULL and combine(y8=None) == NULL and combine(sc=None) == NULL
    assert combine(y=U) == ALIGN and combine(out=U) == ALIGN and combine(y8=U) == ALIGN
    assert combine(T=0, y=None, out=None, y8=None, sc=None) == 0


def test_combine_backward_act8():
    assert combine_bwd(dt=2) == DTYPE
    assert combine_bwd(T=-1) == SHAPE and combine_bwd(d=40) == SHAPE
    assert combine_bwd(k=9, E=64) == SHAPE and combine_bwd(k=3, E=2) == SHAPE
    assert combine_bwd(E=257) == SHAPE and combine_bwd(T=1 << 30, k=4) == SHAPE
    assert combine_bwd(dout=None) == NULL and combine_bwd(sc=None) == NULL
    assert combine_bwd(dy=None) == NULL and combine_bwd(dl=None) == NULL
    assert combine_bwd(dout=U) == ALIGN and combine_bwd(dy=U) == ALIGN and combine_bwd(y8=U) == ALIGN
    assert combine_bwd(T=0, dout=None, y8=None, sc=None, dy=None, dl=None) == 0


def test_backward_act8():
    b, c = moe.BwdDesc(), moe.Act8Saved()
    call = lambda: lib.moe_backward_act8(ctypes.byref(b), ctypes.byref(c), None)
    assert lib.moe_backward_act8(ctypes.byref(b), None, None) == NULL
    assert lib.moe_backward_act8(None, ctypes.byref(c), None) == NULL
    b.dtype, b.d, b.h, b.E, b.k, b.T = BF16, 64, 64, 8, 2, 16
    for n in ("x_perm", "ab", "hp", "topk_gate", "topk_idx", "token_pos", "offsets", "w1", "w2",
              "dout", "dx", "dlogits", "dw1", "dw2", "dy_perm", "dab", "dx_perm"):
        setattr(b, n, F)
    assert call() == NULL                                   # no checkpoints
    c.ab8, c.ab8_scale, c.y8 = F, F, F
    assert call() == NULL
    c.y8_scale, c.ab8 = F, U
    assert call() == ALIGN
    c.ab8, b.hp = F, None                                   # the scratch is needed
    assert call() == NULL
    b.dtype, b.d, b.h = moe.MOE_MXFP8, 128, 128
    for n in ("x", "sorted_token", "w1t", "w1t_scale", "w2t", "w2t_scale", "ws"):
        setattr(b, n, F)
    assert call() == NULL                                   # neither hp nor hp_cols
    b.hp = F
    assert call() == WS
    b.ws_bytes = 1 << 30
    c.y8 = None
    assert call() == NULL


def norm(dt=BF16, T=16, d=64, eps=1e-5, x=F, res=None, ga=F, be=None, y=F, s=None, mean=F, x8=None,
         sc=None):
    return lib.moe_layer_norm(x, dt, res, ga, be, eps, T, d, y, s, mean, F, x8, sc, None)


def test_layer_norm():
    assert norm(dt=2) == DTYPE
    assert norm(T=-1) == SHAPE and norm(T=1 << 31) == SHAPE
    assert norm(d=0) == SHAPE and norm(d=48) == SHAPE and norm(d=16384 + 32) == SHAPE
    for eps in (0.0, -1e-5, float("nan"), 2.0):
        assert norm(eps=eps) == SHAPE
    assert norm(x=None) == NULL and norm(ga=None) == NULL and norm(y=None) == NULL
    assert norm(res=F) == NULL and norm(s=F) == NULL        # residual and sum together
    assert norm(x8=F) == NULL and norm(sc=F) == NULL
    assert norm(x=U) == ALIGN and norm(ga=U) == ALIGN and norm(be=U) == ALIGN
    assert norm(y=U) == ALIGN and norm(res=F, s=U) == ALIGN and norm(x8=U, sc=F) == ALIGN
    assert norm(mean=F + 2) == ALIGN
    assert norm(T=0, x=None, ga=None, y=None) == 0


def norm_bwd(dt=BF16, T=16, d=64, dy=F, x=F, x8=None, sc=None, mean=F, ga=F, dx=F, dg=F, db=F,
             acc=0, ws=F, nb=1 << 20):
    return lib.moe_layer_norm_backward(dy, dt, x, x8, sc, mean, F, ga, None, T, d, dx, dg, db, acc,
                                       ws, nb, None)


def test_layer_norm_backward():
    assert norm_bwd(dt=2) == DTYPE and norm_bwd(acc=2) == DTYPE
    assert norm_bwd(T=-1) == SHAPE and norm_bwd(d=33) == SHAPE
    assert norm_bwd(dy=None) == NULL and norm_bwd(mean=None) == NULL and norm_bwd(dx=None) == NULL
    assert norm_bwd(x=None) == NULL                         # neither x nor its checkpoint
    assert norm_bwd(x8=F, sc=F) == NULL                     # both
    assert norm_bwd(x=None, x8=F) == NULL
    assert norm_bwd(dy=U) == ALIGN and norm_bwd(dx=U) == ALIGN and norm_bwd(ga=U) == ALIGN
    assert norm_bwd(dg=F + 2) == ALIGN and norm_bwd(mean=F + 1) == ALIGN
    assert norm_bwd(ws=None) == NULL and norm_bwd(ws=U) == ALIGN and norm_bwd(nb=16) == WS


def test_layer_norm_backward_workspace():
    size = lib.moe_layer_norm_backward_workspace_size
    assert size(BF16, 0, 64) == 0 and size(7, 16, 64) == 0 and size(BF16, 16, 48) == 0
    assert size(BF16, 1, 64) > 0
    for dt, d in ((BF16, 2048), (F32, 16384), (BF16, 32)):
        assert size(dt, 1 << 20, d) == size(dt, 1 << 30, d) <= 64 << 20    # bounded in T


def test_binding_refuses_what_does_not_fit():
    """CPU tensors, other types, widths and layouts never reach the library."""
    z = torch.zeros
    with pytest.raises(ValueError):
        moe.moe_act8_store(z(4, 64))                                   # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_act8_store(z(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.moe_act8_store(z(4, 40))
    with pytest.raises(ValueError):
        moe.moe_act8_load(z(4, 64, dtype=torch.uint8), z(4, 2, dtype=torch.uint8), torch.float16)
    with pytest.raises(ValueError):
        moe.moe_act8_swiglu(z(4, 96, dtype=torch.uint8), z(4, 3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_layer_norm(z(4, 64), z(64))
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward({}, z(4, 64), z(64))
    with pytest.raises(ValueError):
        moe.moe_combine_act8(z(4, 64), z(2, 2), z(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.moe_combine_backward_act8(z(2, 64), z(4, 64, dtype=torch.uint8),
                                      z(4, 2, dtype=torch.uint8), z(2, 2), z(2, 2), z(2, 2), 8)
    w1, w2 = z(2, 64, 32), z(2, 32, 32)
    with pytest.raises(ValueError):
        moe.MoELayer(w1, w2, 1, recompute=True, act8=True)
    with pytest.raises(ValueError):
        moe.LayerNorm(z(64)).backward(z(4, 64))


def test_calls_go_to_the_tensors_gpu(monkeypatch):
    """A call on a GPU that is not the current one makes it current for the
    call and takes its stream; a refusal raises either way."""
    seen, current = [], [1]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(moe, "_cur_device", lambda: current[0])
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    call = lambda a, stream: seen.append((a, stream, current[0])) or a
    moe._enqueue("f", call, 0, 0)
    moe._enqueue("f", call, 1, 0)
    assert seen == [(0, 100, 0), (0, 101, 1)] and current == [1]
    for index in (0, 1):
        with pytest.raises(moe.MoeError):
            moe._enqueue("f", call, index, moe.MOE_ERR_SHAPE)
    assert current == [1]
