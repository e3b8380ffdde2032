"""The experts with 4-bit weights in plain numpy, in 64 bits: OCP MXFP4
quantisation and the layer's forward on the weights it stands for."""
from __future__ import annotations

import numpy as np

from oracle.train_ops import silu

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def encode(w: np.ndarray):
    """(codes uint8 [rows, cols], scale bytes [rows, cols/32]): per block of 32
    the shared exponent floor(log2 amax) - 2 (-127 at least), elements rounded
    to the nearest E2M1 value, ties to the even code, saturated to 6."""
    rows, cols = w.shape
    b = np.asarray(w, np.float64).reshape(rows, cols // 32, 32)
    amax = np.abs(b).max(axis=2)
    _, e = np.frexp(amax)
    e = np.where(amax == 0, -127, np.maximum(e - 1 - 2, -127))
    v = np.minimum(np.ldexp(np.abs(b), -e[..., None]), 6.0)
    dist = np.abs(v[..., None] - VALUES)
    best = dist.min(axis=-1, keepdims=True)
    near = dist == best                        # one code, or two at a tie
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) == 1, near.argmax(-1), even.argmax(-1)).astype(np.uint8)
    code |= np.signbit(b).astype(np.uint8) << 3
    return code.reshape(rows, cols), (e + 127).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | codes[..., 1::2] << 4


def decode(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    rows, cols = codes.shape
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.ldexp(1.0, scale.astype(int) - 127)
    return (v.reshape(rows, cols // 32, 32) * s[..., None]).reshape(rows, cols)


def experts(x, idx, gate, w1, w2):
    """out [T, d] and its error's first-order weights: the sums of magnitudes
    behind every output (for counting roundings)."""
    x, gate = np.asarray(x, np.float64), np.asarray(gate, np.float64)
    T, k = idx.shape
    h = w2.shape[2]
    u = 2.0 ** -23                             # a matrix unit's fp32 addition, a full step
    out, tol = np.zeros_like(x), np.zeros_like(x)
    for t in range(T):
        for j in range(k):
            a1, a2 = w1[idx[t, j]], w2[idx[t, j]]
            ab, mag = a1 @ x[t], np.abs(a1) @ np.abs(x[t])
            eab = (x.shape[1] + 8) * u * mag
            a, b = ab[:h], ab[h:]
            hid = silu(a) * b
            # |silu'| <= 1.1; exp's argument and roundings; h as two bf16 halves: 2^-16
            eh = 1.1 * eab[:h] * np.abs(b) + np.abs(silu(a)) * eab[h:] + 1.1 * eab[:h] * eab[h:]
            eh += ((10 + 2 * np.abs(a)) * u + 2.0 ** -16) * np.abs(hid)
            y = a2 @ hid
            ey = np.abs(a2) @ eh + (2 * h + 8) * u * (np.abs(a2) @ np.abs(hid))
            out[t] += gate[t, j] * y
            tol[t] += gate[t, j] * (ey + (k + 2) * u * np.abs(y))
    return out, tol
