"""Refusals of the root-mean-square norm, the MXFP8 dequantisation and the
gradients' norm and clipping (no GPU needed): each bad argument gives the
documented status before anything is enqueued, and the binding raises on
tensors that do not fit."""
import ctypes
import weakref

import pytest
import torch

import routing_grouped_gemm_router_amd as moe

F = 0x100000          # never dereferenced: validation fails first
U = F + 4             # not 16-byte aligned
NULL, SHAPE, DTYPE, ALIGN, WS = 1, 2, 3, 4, 5
BF16, F32 = moe.MOE_BF16, moe.MOE_F32
lib = moe.lib()


def _rms(x=F, dt=BF16, res=None, ga=F, eps=1e-6, T=4, d=64, y=F, sm=None, rstd=F, yq=None, yqs=None,
         x8=None, x8s=None):
    return lib.moe_rms_norm(x, dt, res, ga, eps, T, d, y, sm, rstd, yq, yqs, x8, x8s, None)


@pytest.mark.parametrize("kw,st", [
    (dict(dt=moe.MOE_MXFP8), DTYPE), (dict(dt=9), DTYPE), (dict(d=48), SHAPE), (dict(d=0), SHAPE),
    (dict(d=16384 + 32), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(eps=0.0), SHAPE),
    (dict(eps=2.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(x=None), NULL), (dict(ga=None), NULL),
    (dict(y=None), NULL), (dict(res=F), NULL), (dict(sm=F), NULL), (dict(yq=F), NULL), (dict(yqs=F), NULL),
    (dict(x8=F), NULL), (dict(x8s=F), NULL), (dict(x=U), ALIGN), (dict(y=U), ALIGN), (dict(ga=U), ALIGN),
    (dict(yq=U, yqs=F), ALIGN), (dict(x8=U, x8s=F), ALIGN), (dict(res=U, sm=F), ALIGN),
    (dict(res=F, sm=U), ALIGN), (dict(rstd=F + 2), ALIGN), (dict(T=0, x=None, y=None, ga=None), 0),
])
def test_rms_norm(kw, st):
    assert _rms(**kw) == st


def _rms_bwd(dy=F, dt=BF16, x=F, x8=None, x8s=None, rstd=F, ga=F, ds=None, T=4, d=64, dx=F, dg=F, acc=0,
             ws=F, wsb=1 << 20):
    return lib.moe_rms_norm_backward(dy, dt, x, x8, x8s, rstd, ga, ds, T, d, dx, dg, acc, ws, wsb, None)


@pytest.mark.parametrize("kw,st", [
    (dict(dt=2), DTYPE), (dict(acc=2), DTYPE), (dict(d=33), SHAPE), (dict(T=-1), SHAPE), (dict(dy=None), NULL),
    (dict(x=None), NULL), (dict(x8=F, x8s=F), NULL), (dict(x=None, x8=F), NULL), (dict(rstd=None), NULL),
    (dict(ga=None), NULL), (dict(dx=None), NULL), (dict(dy=U), ALIGN), (dict(dx=U), ALIGN), (dict(ds=U), ALIGN),
    (dict(dg=F + 1), ALIGN), (dict(rstd=F + 2), ALIGN), (dict(wsb=16), WS), (dict(ws=None), NULL),
    (dict(ws=U), ALIGN),
])
def test_rms_norm_backward(kw, st):
    assert _rms_bwd(**kw) == st


def test_rms_workspace():
    n = moe.moe_rms_norm_backward_workspace_size
    assert n(BF16, 16384, 2048) == 512 * 2048 * 4 and n(F32, 1, 32) == 32 * 4
    assert n(BF16, 4, 48) == 0 and n(7, 4, 64) == 0 and n(F32, 0, 64) == 0


@pytest.mark.parametrize("args,st", [
    ((F, F, moe.MOE_MXFP8, 4, 64, F, None), DTYPE), ((F, F, F32, 4, 33, F, None), SHAPE),
    ((F, F, F32, -1, 64, F, None), SHAPE), ((F, F, F32, 4, 1 << 20, F, None), SHAPE),
    ((None, F, F32, 4, 64, F, None), NULL), ((F, None, F32, 4, 64, F, None), NULL),
    ((F, F, F32, 4, 64, None, None), NULL), ((F, F, F32, 4, 64, U, None), ALIGN),
    ((U, F, F32, 4, 64, F, None), ALIGN), ((None, None, F32, 0, 64, None, None), 0),
])
def test_dequantize(args, st):
    assert lib.mxfp8_dequantize(*args) == st


def _grads(*items):
    """items: (data, out, n, dtype)."""
    v = [x or 0 for it in items for x in it]
    return (ctypes.c_int64 * max(len(v), 1))(*v)


def _clip(items, n=None, max_norm=1.0, norm=F, ws=F, wsb=1 << 30):
    return lib.moe_clip_grad_norm(_grads(*items), len(items) if n is None else n, max_norm, norm, ws, wsb, None)


A = (F, 0, 8, F32)    # 32 bytes


@pytest.mark.parametrize("items,st", [
    ([(F, 0, 8, moe.MOE_MXFP8)], DTYPE), ([(F, 0, 8, 7)], DTYPE), ([(F, 0, -1, F32)], SHAPE),
    ([(F, 0, 1 << 56, F32)], SHAPE), ([(0, 0, 8, F32)], NULL), ([(0, F, 8, F32)], NULL),
    ([(F + 2, 0, 8, F32)], ALIGN), ([(F + 1, 0, 8, BF16)], ALIGN), ([(F, F + 0x102, 8, F32)], ALIGN),
    ([A, A], SHAPE),                                       # the same tensor twice
    ([A, (F + 28, 0, 8, F32)], SHAPE),                     # one element in common
    ([(F + 28, 0, 8, F32), A], SHAPE),
    ([A, (F + 30, 0, 8, BF16)], SHAPE),
    ([(F, F + 4, 8, F32)], SHAPE),                         # out over its own data, one element on
    ([(F + 4, F, 8, F32)], SHAPE),
    ([(F, F + 0x100, 8, F32), (F + 0x80, F + 0x100, 8, F32)], SHAPE),    # two outs in one place
    ([(F, F + 0x80, 8, F32), (F + 0x80, F + 0x100, 8, F32)], SHAPE),     # an out over another's data
    ([(F, F + 0x80, 8, F32), (F + 0x90, 0, 8, F32)], SHAPE),
])
def test_clip_refuses(items, st):
    assert _clip(items) == st
    assert lib.moe_grad_clip(_grads(*items), len(items), F, 1.0, None) == st


def test_clip_refuses_scalars():
    assert _clip([A], max_norm=-1.0) == SHAPE and _clip([A], max_norm=float("nan")) == SHAPE
    assert lib.moe_grad_clip(_grads(A), 1, F, float("nan"), None) == SHAPE
    assert _clip([A], n=-1) == SHAPE and _clip([A], n=moe.MOE_GRAD_MAX + 1) == SHAPE
    assert _clip([A], norm=None) == NULL and _clip([A], norm=F + 2) == ALIGN
    assert _clip([A], ws=None) == NULL and _clip([A], ws=U) == ALIGN and _clip([A], wsb=16) == WS
    assert lib.moe_clip_grad_norm(None, 1, 1.0, F, F, 1 << 20, None) == NULL
    assert lib.moe_grad_clip(_grads(A), 1, None, 1.0, None) == NULL
    assert lib.moe_grad_norm(_grads(A), 1, None, F, 1 << 20, None) == NULL
    assert lib.moe_grad_norm(_grads(A), 1, F, F, 100, None) == WS
    assert lib.moe_grad_norm(_grads((F + 2, 0, 4, F32)), 1, F, F, 1 << 20, None) == ALIGN


def test_norm_workspace():
    n = moe.moe_grad_norm_workspace_size
    assert n(0) == 0 and n(1) == n(64) == 16384 and n(65) == 32768 and n(-1) == 0 and n(4097) == 0


def test_binding_refuses():
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_rms_norm(x, w)
    for fn in (moe.moe_grad_norm, lambda g: moe.moe_clip_grad_norm(g, 1.0),
               lambda g: moe.moe_grad_clip(g, x, 1.0)):
        with pytest.raises(ValueError, match="at least one"):
            fn([])
        with pytest.raises(ValueError, match=r"grads\[0\]: expected a contiguous f32 or bf16 tensor on a GPU"):
            fn([x])
    with pytest.raises(ValueError, match="out: expected 1 tensors"):
        moe.moe_clip_grad_norm([x], 1.0, out=[x, x])
    with pytest.raises(ValueError, match="GPU"):
        moe.mxfp8_dequantize(x.to(torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))


@pytest.mark.parametrize("call", ["norm", "clip", "clip into others", "by a norm"])
def test_tensors_live_until_the_call(monkeypatch, call):
    """Tensors that only an iterator hands out are still there when the kernels
    are enqueued: their memory must not have gone to the workspace before."""
    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    refs, alive = [], []

    def tensors():
        for _ in range(5):
            t = torch.ones(64).as_subclass(OnGpu)
            refs.append(weakref.ref(t))
            yield t

    monkeypatch.setattr(moe, "_t_gpu", lambda t: 0)
    monkeypatch.setattr(moe, "_enqueue", lambda *a: alive.extend(r() is not None for r in refs))
    if call == "norm":
        moe.moe_grad_norm(tensors())
    elif call == "clip":
        moe.moe_clip_grad_norm(tensors(), 1.0)
    elif call == "clip into others":
        moe.moe_clip_grad_norm(tensors(), 1.0, out=tensors())
    else:
        moe.moe_grad_clip(tensors(), torch.ones(()).as_subclass(OnGpu), 1.0, out=tensors())
    assert alive and all(alive)
