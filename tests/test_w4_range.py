"""The 4-bit products at the ends of the number range, through each of their
kernels: H' beyond bf16's largest value, infinities, the first and the last
scale bytes; and the quantisation there."""
import numpy as np
import pytest
import torch

import oracle.w4 as w4
import synth
from helpers import dev, to_np

import routing_grouped_gemm_router_amd as moe

pytestmark = pytest.mark.gpu

# T, d, h, E, k: the down product by token; both products by tiles of 8 rows;
# the wide kernel for gate and up; for down
KERNELS = [(1, 64, 64, 4, 1), (20, 96, 64, 2, 1), (400, 448, 2048, 16, 1), (200, 4128, 160, 4, 4)]


def _codes(E, rows, cols, seed):
    rng = np.random.default_rng(seed)
    return rng.integers(0, 16, (E * rows, cols)).astype(np.uint8)


class Weights:
    """Codes and scale bytes of W1 and W2, to be changed before `cuda`."""

    def __init__(self, d, h, E, seed, scale1=127, scale2=127):
        self.E, self.d, self.h = E, d, h
        self.c1, self.c2 = _codes(E, 2 * h, d, seed), _codes(E, d, h, seed + 1)
        self.s1 = np.full((E * 2 * h, d // 32), scale1, np.uint8)
        self.s2 = np.full((E * d, h // 32), scale2, np.uint8)

    def view1(self, a):                                    # [E, 2 (a, b), h, ..]
        return a.reshape(self.E, 2, self.h, -1)

    def cuda(self):
        cu = lambda a, *sh: torch.from_numpy(np.ascontiguousarray(a)).cuda().view(*sh)
        E, d, h = self.E, self.d, self.h
        return (cu(w4.pack(self.c1), E, 2 * h, d // 2), cu(self.s1, E, 2 * h, d // 32),
                cu(w4.pack(self.c2), E, d, h // 2), cu(self.s2, E, d, h // 32))

    def values(self):
        return (w4.decode(self.c1, self.s1).reshape(self.E, 2 * self.h, self.d),
                w4.decode(self.c2, self.s2).reshape(self.E, self.d, self.h))


def _route(T, E, k):
    return moe.moe_route(dev(synth.normal((T, E), 5, 0, 1.0), torch.float32), k)


def _check(out, x, r, w):
    """Within the roundings counted by the oracle, and half a step of bf16."""
    ref, tol = w4.experts(to_np(x), to_np(r["topk_idx"]), to_np(r["topk_gate"]), *w.values())
    got = to_np(out).astype(np.float64)
    assert np.isfinite(ref).all()
    bad = ~(np.abs(got - ref) <= tol + torch.finfo(torch.bfloat16).eps / 2 * (np.abs(ref) + tol))
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("T,d,h,E,k", KERNELS)
@pytest.mark.parametrize("last", [False, True])
def test_hidden_beyond_bf16(T, d, h, E, k, last):
    """H' = (2^8 - 1)(2^8 + 1) 2^112 = 2^128 - 2^112 is finite in fp32 and rounds
    to infinity in bf16; in another token it is infinite in fp32 too. The hidden
    unit is the first or the last one, its inputs the first or last three."""
    w = Weights(d, h, E, T + d, 120, 120)
    unit, at = (h - 1, (d - 1, d - 2, d - 3)) if last else (0, (0, 1, 2))
    c1, s1 = w.view1(w.c1), w.view1(w.s1)
    c1[..., list(at)] = 0                                  # nothing else reads these inputs
    c1[:, :, unit] = 0
    s1[:, :, unit] = 127 + 56
    c1[:, 0, unit, at[0]] = 2                              # a = 2^56 x[at[0]]
    c1[:, 1, unit, at[1]] = c1[:, 1, unit, at[2]] = 2      # b = 2^56 (x[at[1]] + x[at[2]])
    w.c2[:, unit] = 2 + w.c2[:, unit] % 6                  # positive
    w.s2[:, unit // 32] = 27                               # 2^-100
    x = dev(synth.normal((T, d), 5, 1, 1.0), torch.bfloat16)
    x[:, list(at)] = 0
    t = T // 2
    x[t, at[0]], x[t, at[1]], x[t, at[2]] = 255, 256, 1
    r = _route(T, E, k)
    args = w.cuda()
    out = moe.moe_w4_experts(x, r, *args)
    assert to_np(out[t]).min() > 2.0 ** 26
    _check(out, x, r, w)
    over = x.clone()
    over[t, at[0]] = 2.0 ** 20
    got = moe.moe_w4_experts(over, r, *args)
    assert (got[t] == float("inf")).all()
    rest = torch.arange(T, device="cuda") != t
    assert torch.equal(got[rest], out[rest])


@pytest.mark.parametrize("T,d,h,E,k", KERNELS)
@pytest.mark.parametrize("last", [False, True])
def test_infinite_input(T, d, h, E, k, last):
    """An infinity in x, met by positive weights alone: infinite a, b, H' and
    out, no NaN from the places past a row's end."""
    w = Weights(d, h, E, T + d, 120, 120)
    c = d - 1 if last else 0
    w.c1[:, c] = 1 + w.c1[:, c] % 7
    w.c2[:] = 1 + w.c2 % 7
    x = dev(synth.normal((T, d), 5, 1, 1.0), torch.bfloat16)
    r = _route(T, E, k)
    args = w.cuda()
    out = moe.moe_w4_experts(x, r, *args)
    _check(out, x, r, w)
    over, t = x.clone(), T // 2
    over[t, c] = float("inf")
    got = moe.moe_w4_experts(over, r, *args)
    assert (got[t] == float("inf")).all()
    rest = torch.arange(T, device="cuda") != t
    assert torch.equal(got[rest], out[rest])


@pytest.mark.parametrize("T,d,h,E,k", KERNELS)
@pytest.mark.parametrize("s1,s2,xe", [(0, 127, 119), (1, 127, 118), (252, 127, -117), (127, 0, 54),
                                      (127, 1, 53), (127, 252, -59)])
def test_end_scales(T, d, h, E, k, s1, s2, xe):
    """Scale bytes at the ends: elements of code 2^(s - 127), from 2^-128, a
    subnormal number, to 6 2^125. x is scaled so that a, b, H' and out are
    normal numbers."""
    w = Weights(d, h, E, T + d, s1, s2)
    x = dev(np.clip(synth.normal((T, d), 5, 1, 1.0), -3, 3) * 2.0 ** xe, torch.bfloat16)
    r = _route(T, E, k)
    out = moe.moe_w4_experts(x, r, *w.cuda())
    assert float(out.abs().max()) > 2.0 ** -60
    _check(out, x, r, w)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_quantize_at_the_ends(dt):
    """Blocks whose largest magnitude is at the ends of fp32's range: scale
    byte 0 from 2^-125 down, elements down to the smallest subnormals; 252 at
    the top."""
    rng = np.random.default_rng(3)
    tops = [2.0 ** -124, 2.0 ** -125, 1.99 * 2.0 ** -125, 2.0 ** -126, 1.5 * 2.0 ** -126, 2.0 ** -127,
            1.5 * 2.0 ** -127, 2.0 ** -128, 2.0 ** -129, 2.0 ** -130, 2.0 ** -133, 2.0 ** -149,
            2.0 ** 127, 1.5 * 2.0 ** 127, 3.38e38]
    part = np.r_[1, -1, np.array([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12]) / 12, -np.arange(1, 7) / 8]
    x = np.zeros((len(tops), 64), np.float32)
    for i, top in enumerate(tops):
        x[i, :20] = (top * part).astype(np.float32)
        x[i, 32:] = (top * np.r_[1, rng.uniform(-1, 1, 31)]).astype(np.float32)
    t = torch.from_numpy(x).to(dt)
    q, s = moe.moe_w4_quantize(t.cuda())
    c, e = w4.encode(t.float().numpy())
    assert np.array_equal(to_np(s), e)
    assert e.min() == 0 and e.max() == 252
    got = np.stack([to_np(q) & 15, to_np(q) >> 4], -1).reshape(x.shape)
    zero = (c & 7) == 0                                    # a zero's sign says nothing
    assert np.array_equal(np.where(zero, got & 7, got), np.where(zero, 0, c))
