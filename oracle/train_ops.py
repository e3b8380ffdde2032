"""The 8-bit activation checkpoints and the layer norm in plain numpy, in 64
bits: what the library's moe_act8_*, moe_combine_act8,
moe_combine_backward_act8 and moe_layer_norm* compute, from their formulas.

Arrays that hold bf16 data are float32 / float64 arrays of bf16 values;
rounding a result to the storage type is left to the caller."""
from __future__ import annotations

import numpy as np


def act8_encode(x: np.ndarray):
    """(codes int8 [rows, cols], scale bytes uint8 [rows, cols/32]) of x, by the
    definition of OCP MXINT8: per 32 elements the scale 2^floor(log2 amax)
    (2^-127 at least), elements in multiples of a 64th of it, rounded to
    nearest even, symmetric range. A block with a NaN or an infinity: scale
    byte 255, zeros."""
    rows, cols = x.shape
    b = np.asarray(x, np.float64).reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    _, e = np.frexp(amax)                           # amax = m 2^e, 1/2 <= m < 1
    e = np.where(amax == 0, -127, np.maximum(e - 1, -127))
    c = np.clip(np.rint(np.ldexp(b, (6 - e)[..., None])), -127, 127)
    c = np.where(bad[..., None], 0, c).astype(np.int8).reshape(rows, cols)
    return c, np.where(bad, 255, e + 127).astype(np.uint8)


def act8_decode(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The values that a checkpoint stands for (float64)."""
    rows, cols = codes.shape
    c = codes.view(np.int8).astype(np.float64).reshape(rows, cols // 32, 32)
    v = np.ldexp(c, scale.astype(np.int64)[..., None] - 133)
    return np.where((scale == 255)[..., None], np.nan, v).reshape(rows, cols)


def act8(x: np.ndarray) -> np.ndarray:
    """x as its checkpoint gives it back."""
    return act8_decode(*act8_encode(x))


def silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


def swiglu_hidden(ab: np.ndarray) -> np.ndarray:
    a, b = np.split(np.asarray(ab, np.float64), 2, axis=1)
    return silu(a) * b


def layer_norm(s, gamma, beta, eps):
    """(y, mean, rstd) over the rows of s."""
    s = np.asarray(s, np.float64)
    mean = s.mean(axis=1)
    rstd = 1 / np.sqrt(((s - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (s - mean[:, None]) * rstd[:, None] * np.asarray(gamma, np.float64)
    return (y if beta is None else y + np.asarray(beta, np.float64)), mean, rstd


def layer_norm_backward(s, mean, rstd, dy, gamma, dsum=None):
    """(dx, dgamma, dbeta) with the given statistics."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (s - np.asarray(mean, np.float64)[:, None]) * r
    g = dy * np.asarray(gamma, np.float64)
    dx = r * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def rms_norm(s, gamma, eps):
    """Root-mean-square norm of rows s [T, d]: y = s rstd gamma, rstd."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).sum(1) / s.shape[1] + eps)
    return s * rstd[:, None] * np.asarray(gamma, np.float64), rstd


def rms_norm_backward(s, rstd, dy, gamma, dsum=None):
    """dx (the gradient of s, plus dsum), dgamma."""
    s, dy, r = (np.asarray(a, np.float64) for a in (s, dy, np.asarray(rstd)[:, None]))
    xh, g = s * r, dy * np.asarray(gamma, np.float64)
    dx = r * (g - xh * (g * xh).mean(1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * xh).sum(0)


def combine(y, gate, token_pos):
    """out[t] = sum_j gate[t, j] y[token_pos[t, j]]; a negative position adds nothing."""
    keep = token_pos >= 0
    rows = np.where(keep[..., None], np.asarray(y, np.float64)[np.maximum(token_pos, 0)], 0.0)
    return (np.asarray(gate, np.float64)[..., None] * rows).sum(axis=1)


def combine_backward(dout, y, gate, topk_idx, token_pos, E):
    """dict of dy_perm (rows that no position names: NaN), dlogits, dgate."""
    dout, y, gate = (np.asarray(a, np.float64) for a in (dout, y, gate))
    T, k = token_pos.shape
    dy = np.full((y.shape[0], dout.shape[1]), np.nan)
    dgate = np.zeros((T, k))
    dlogits = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            p = token_pos[t, j]
            if p >= 0:
                dgate[t, j] = dout[t] @ y[p]
                dy[p] = gate[t, j] * dout[t]
        for j in range(k):
            dlogits[t, topk_idx[t, j]] = gate[t, j] * (gate[t] * (dgate[t, j] - dgate[t])).sum()
    return dict(dy_perm=dy, dlogits=dlogits, dgate=dgate)
