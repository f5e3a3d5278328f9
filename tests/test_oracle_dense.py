"""Pins of the oracle of dense layers (oracle/dense.py): gradients against central differences of its own forward
functions, closed forms, hand values."""
import numpy as np
import pytest

from oracle import dense as OD


def _differences(f, x, step=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        d[i] = (f(hi) - f(lo)) / (2 * step)
    return d


def test_layernorm_by_hand():
    # deviations (-1, 1) of mean 3 have variance 1
    _, y = OD.add_layernorm(np.array([[2.0, 4.0]]), None, np.array([1.0, 2.0]), np.array([0.5, 0.0]), 0.0)
    assert np.allclose(y, [[-0.5, 2.0]], atol=1e-15)
    # the residual is added and rounded to bf16 first: 1 + 2^-9 rounds to 1
    h, _ = OD.add_layernorm(np.array([[1.0, 8.0]]), np.array([[2.0 ** -9, 1.0]]), np.ones(2), None, 1e-5)
    assert np.array_equal(h, [[1.0, 9.0]])
    # a row of equal values is the bias
    _, y = OD.add_layernorm(np.full((1, 5), 7.0), None, np.ones(5), np.arange(5.0), 1e-5)
    assert np.array_equal(y, np.arange(5.0)[None])


def test_layernorm_gradients():
    g = np.random.default_rng(1)
    x, w, dy, dh = g.standard_normal((3, 10)), g.standard_normal(10), g.standard_normal((3, 10)), g.standard_normal((3, 10))
    dx, dw, db, mag, wm, bm = OD.layernorm_backward(dy, x, w, 1e-3, dh)
    f = lambda x_, w_, b_: (OD.add_layernorm(x_, None, w_, b_, 1e-3)[1] * dy).sum() + (x_ * dh).sum()
    b = np.zeros(10)
    assert np.allclose(dx, _differences(lambda v: f(v, w, b), x), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: f(x, v, b), w), atol=1e-7)
    assert np.allclose(db, _differences(lambda v: f(x, w, v), b), atol=1e-7)
    assert (mag >= np.abs(dx) - 1e-12).all() and (wm >= np.abs(dw)).all() and (bm >= np.abs(db)).all()
    # a constant added to a row, and a factor without eps, change nothing: dx is orthogonal to both
    dx0 = OD.layernorm_backward(dy, x, w, 0.0)[0]
    assert np.allclose(dx0.sum(1), 0, atol=1e-12)
    assert np.allclose((dx0 * (x - x.mean(1, keepdims=True))).sum(1), 0, atol=1e-12)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_gated_gradients(act):
    g = np.random.default_rng(2)
    gg, u, dh = g.standard_normal((4, 9)) * 2, g.standard_normal((4, 9)), g.standard_normal((4, 9))
    d, mag = OD.gated_backward(dh, gg, u, act)
    f = lambda a, b: (OD.activation(a, act) * b * dh).sum()
    num = np.concatenate([_differences(lambda v: f(v, u), gg), _differences(lambda v: f(gg, v), u)], 1)
    assert np.allclose(d, num, atol=1e-7) and (mag >= np.abs(d) - 1e-12).all()


def test_activations_far_out():
    v = np.array([-30.0, -12.0, 0.0, 40.0])
    # erfc(z) = exp(-z^2) / (z sqrt pi) (1 - 1 / (2 z^2) + ..)
    z = 12 / np.sqrt(2)
    tail = -6.0 * np.exp(-z * z) / (z * np.sqrt(np.pi)) * (1 - 1 / (2 * z * z) + 3 / (4 * z ** 4))
    assert np.isclose(OD.activation(v, "gelu")[1], tail, rtol=1e-4)
    assert OD.activation(v, "silu")[0] == -30 / (1 + np.exp(30.0))
    for act in ("silu", "gelu", "gelu_tanh"):
        a, s = OD.activation(v, act), OD.activation_slope(v, act)[0]
        assert a[2] == 0 and a[3] == 40 and s[2] == 0.5 and abs(s[3] - 1) < 1e-12 and abs(s[0]) < 1e-10 and (a[:2] <= 0).all() and a[1] < 0


def test_gated_by_hand():
    h, g, u = OD.gated(np.array([[1.0, 2.0]]), np.array([[1.0, -1.0, 3.0, 0.0], [0.5, 0.0, 0.0, 1.0]]), np.array([0.0, 4.0, 1.0, 1.0]), "relu")
    assert np.array_equal(g, [[2.0, 3.0]]) and np.array_equal(u, [[4.0, 3.0]]) and np.array_equal(h, [[8.0, 9.0]])


def test_lora_by_hand():
    x = np.arange(8.0).reshape(4, 2)
    a, b = np.array([[[1.0, 0.0]], [[0.0, 2.0]]]), np.array([[[1.0], [0.0], [2.0]], [[0.0], [1.0], [0.0]]])
    y0 = np.full((4, 3), 9.0)
    y, mag = OD.lora(x, a, b, [0.5, 1.0], [1, 5, 0], [-3, 1, 2, 3], np.ones((4, 3)), y0)
    # row 0: 2 x[1] into column 1; row 1: no adapter; row 2: x[0] / 2 into columns 0 and 2; row 3: outside
    assert np.array_equal(y, [[1, 3, 1], [1, 1, 1], [3, 1, 5], [9, 9, 9]])
    assert np.array_equal(mag, [[0, 2, 0], [0, 0, 0], [2, 0, 4], [0, 0, 0]])
    y, _ = OD.lora(x, a, b, [1.0, 1.0], [0, 0, 1, -1], None, None, y0)
    assert np.array_equal(y, [[0, 0, 0], [2, 0, 4], [0, 10, 0], [0, 0, 0]])
