"""The plain 64-bit forms of the 8-bit checkpoints and of the layer norm:
closed forms, bounds and difference quotients (CPU)."""
import numpy as np
import pytest

import oracle.train_ops as ops


def test_act8_closed_forms():
    x = np.zeros((1, 64))
    x[0, :6] = [1.0, 0.5, -0.25, 1 / 64, 1.5 / 64, 2.5 / 64]       # amax 1: step 1/64
    x[0, 32:38] = [1.999, -1.999, 126.5 / 64, 127.5 / 64, -0.5 / 64, 0.51 / 64]
    c, s = ops.act8_encode(x)
    assert s.tolist() == [[127, 127]]
    assert c[0, :6].tolist() == [64, 32, -16, 1, 2, 2]              # ties to even
    assert c[0, 32:38].tolist() == [127, -127, 126, 127, 0, 1]      # the clamp
    v = ops.act8_decode(c, s)
    assert v[0, 0] == 1.0 and v[0, 32] == 127 / 64


def test_act8_scale_range():
    x = np.zeros((5, 32))
    x[1, 3] = 2.0 ** -149                     # fp32's smallest subnormal: below half the smallest step
    x[2, 3] = 2.0 ** -127                     # subnormal: scale byte 0, step 2^-133
    x[3, 3] = 2.0 ** 127
    x[4, 3] = np.inf
    c, s = ops.act8_encode(x)
    assert s[:, 0].tolist() == [0, 0, 0, 254, 255]
    assert c[:, 3].tolist() == [0, 0, 64, 64, 0]
    v = ops.act8_decode(c, s)
    assert v[2, 3] == 2.0 ** -127 and v[3, 3] == 2.0 ** 127
    assert np.isnan(v[4]).all()


@pytest.mark.parametrize("scale", [1e-3, 1.0, 1e5])
def test_act8_error_bound(scale):
    """Half a step of the block's power of two over 64; a whole one where the clamp took part."""
    x = np.random.default_rng(0).normal(size=(50, 320)) * scale
    _, s = ops.act8_encode(x)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 133), 32, axis=1)
    err = np.abs(ops.act8(x) - x)
    top = np.abs(x) > 127.5 * step
    assert (err[~top] <= step[~top] / 2).all() and (err[top] <= step[top]).all()
    assert np.array_equal(ops.act8(ops.act8(x)), ops.act8(x))


def test_layer_norm_closed_form():
    s = np.array([[1.0, 2.0, 3.0, 4.0], [5.0, 5.0, 5.0, 5.0]])
    y, mean, rstd = ops.layer_norm(s, np.ones(4), np.full(4, 0.5), 1e-6)
    assert np.allclose(mean, [2.5, 5.0]) and np.allclose(rstd, [1 / np.sqrt(1.25 + 1e-6), 1e3])
    assert np.allclose(y[0] - 0.5, (s[0] - 2.5) / np.sqrt(1.25 + 1e-6)) and np.allclose(y[1], 0.5)


def test_layer_norm_gradient_by_differences():
    rng = np.random.default_rng(1)
    T, d, eps = 3, 8, 1e-3
    s, dy, ds = rng.normal(size=(3, T, d))
    ga, be = rng.normal(size=(2, d))
    loss = lambda s_, g_, b_: (ops.layer_norm(s_, g_, b_, eps)[0] * dy).sum() + (s_ * ds).sum()
    _, mean, rstd = ops.layer_norm(s, ga, be, eps)
    dx, dg, db = ops.layer_norm_backward(s, mean, rstd, dy, ga, ds)
    h = 1e-5                                   # central differences: error O(h^2) ~ 1e-10 of O(1) terms
    for _ in range(4):
        v, vg, vb = rng.normal(size=(T, d)), rng.normal(size=d), rng.normal(size=d)
        num = (loss(s + h * v, ga + h * vg, be + h * vb) - loss(s - h * v, ga - h * vg, be - h * vb)) / (2 * h)
        assert abs(num - ((dx * v).sum() + dg @ vg + db @ vb)) <= 1e-7 * max(1, abs(num))


def test_combine_gradient_by_differences():
    """The combine's and the router's gradient against differences of the
    output through softmax gates, the selection held fixed."""
    rng = np.random.default_rng(2)
    T, k, E, d = 4, 3, 6, 5
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    pos = rng.permutation(T * k).reshape(T, k)
    y, dout, logits = rng.normal(size=(T * k, d)), rng.normal(size=(T, d)), rng.normal(size=(T, E))

    def gates(lg):
        e = np.exp(np.take_along_axis(lg, idx, 1))
        return e / e.sum(1, keepdims=True)

    b = ops.combine_backward(dout, y, gates(logits), idx, pos, E)
    loss = lambda y_, lg: (ops.combine(y_, gates(lg), pos) * dout).sum()
    h = 1e-5
    for _ in range(4):
        vy, vl = rng.normal(size=y.shape), rng.normal(size=logits.shape)
        num = (loss(y + h * vy, logits + h * vl) - loss(y - h * vy, logits - h * vl)) / (2 * h)
        assert abs(num - ((b["dy_perm"] * vy).sum() + (b["dlogits"] * vl).sum())) <= 1e-7 * max(1, abs(num))


def test_combine_dropped_slot():
    y, dout = np.ones((2, 4)), np.ones((1, 4))
    gate, idx, pos = np.array([[0.75, 0.25]]), np.array([[2, 0]]), np.array([[1, -1]])
    assert np.allclose(ops.combine(y, gate, pos), 0.75)
    b = ops.combine_backward(dout, y, gate, idx, pos, 3)
    assert b["dgate"].tolist() == [[4.0, 0.0]] and np.isnan(b["dy_perm"][0]).all()
    assert np.allclose(b["dlogits"], [[-0.75, 0, 0.75]])
