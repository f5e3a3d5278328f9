"""Pins of oracle/layer.py: gradients against central differences of the forward functions, closed
forms and hand values."""
import numpy as np
import pytest

from oracle import codec, layer, mx


def _differences(f, x, step=1e-5):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        g[i] = (f(hi) - f(lo)) / (2 * step)
    return g


def _close(a, b, tol=1e-7):
    # central differences with step 1e-5 in float64: truncation ~ step^2, rounding ~ 1e-16 / step
    assert np.abs(a - b).max() <= tol * max(1.0, np.abs(b).max()), np.abs(a - b).max()


def test_rmsnorm_hand_values():
    h, y = layer.add_rmsnorm(np.array([[3.0, 4.0]]), None, np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    # the sum is rounded to bf16 before it is normalised: 1 + 2^-9 -> 1
    h, _ = layer.add_rmsnorm(np.array([[1.0, 2.0]]), np.array([[2.0 ** -9, 0.0]]), np.ones(2), 1e-6)
    assert np.array_equal(h, [[1.0, 2.0]])


def test_rmsnorm_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    h, w, dy, dh = (rng.standard_normal(s) for s in ((3, 8), (8,), (3, 8), (3, 8)))
    dx, dw, _, _ = layer.rmsnorm_backward(dy, h, w, 1e-3, dh)
    _close(dx, _differences(lambda v: (layer.add_rmsnorm(v, None, w, 1e-3)[1] * dy).sum() + (v * dh).sum(), h))
    _close(dw, _differences(lambda v: (layer.add_rmsnorm(h, None, v, 1e-3)[1] * dy).sum(), w))


@pytest.mark.parametrize("name,at", [("relu", [(-1.0, 0.0), (2.0, 2.0)]), ("silu", [(0.0, 0.0), (1.0, 0.7310585786300049)]),
                                     ("gelu", [(1.0, 0.8413447460685429), (-1.0, -0.15865525393145707)]),
                                     ("gelu_tanh", [(1.0, 0.8411919906082768)]), ("none", [(-3.0, -3.0)])])
def test_activation_hand_values(name, at):
    for v, want in at:
        assert abs(layer.activation(np.array([v]), name)[0] - want) < 1e-15


def test_linear_scales_and_short_block():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 256)), rng.standard_normal((256, 256))
    xq, xs = codec.quant_rows_128(x)
    wq, ws = codec.quant_blocks_128(w)
    xv, wv = layer.dequant_linear(xq, xs, wq, ws, False)
    assert np.array_equal(xv, codec.dequant_rows_128(xq, xs)) and np.array_equal(wv, codec.dequant_blocks_128(wq, ws))
    _, short = layer.dequant_linear(xq, xs, wq[:, :144], ws, False)
    assert np.array_equal(short, wv[:, :144])
    xq, xs = mx.quant_rows_32(x)
    wq, ws = mx.quant_weight_k32(w, mx.FMT_E4M3)
    xv, wv = layer.dequant_linear(xq, xs, wq, ws, True)
    assert np.array_equal(xv, mx.dequant_rows_32(xq, xs)) and np.array_equal(wv, mx.dequant_weight_k32(wq, ws, mx.FMT_E4M3))
    onehot = np.zeros((256, 1))
    onehot[7] = 1.0
    assert np.array_equal(layer.linear(xv, onehot, np.array([1.5]), "none", np.full((3, 1), 2.0))[0], xv[:, 7:8] + 3.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_closed_forms(scoring):
    # uniform probabilities and any counts: sum_e E c_e / (k T) / E = 1
    ids = np.array([[0, 1], [0, 2], [0, 3]])
    losses, counts, mean = layer.balance_loss(np.zeros((3, 4)), ids, 2, scoring, 0.5, 0.25)
    assert np.allclose(losses, [0.5 + 0.25 * np.log(4) ** 2, 0.5, 0.25 * np.log(4) ** 2])
    assert counts.tolist() == [[3, 1, 1, 1]] and np.allclose(mean, 0.25)
    # an empty sequence and padding change nothing but the empty sequence's zero rows
    l = np.random.default_rng(3).standard_normal((5, 4))
    i5 = np.array([[0, 1]] * 5)
    whole = layer.balance_loss(l[:3], i5[:3], 2, scoring, 0.5, 0.25)
    parts = layer.balance_loss(l, i5, 2, scoring, 0.5, 0.25, [0, 0, 3])
    assert np.allclose(whole[0], parts[0]) and parts[1][0].sum() == 0 and np.array_equal(whole[1][0], parts[1][1])
    # a row without a live logit adds nothing
    l[1] = -np.inf
    losses, _, mean = layer.balance_loss(l[:3], i5[:3], 2, "softmax", 0.0, 1.0)
    lse = np.log(np.exp(l[[0, 2]]).sum(1))
    assert np.isclose(losses[2], (lse ** 2).sum() / 3) and np.isclose(mean.sum(), 2 / 3)


@pytest.mark.parametrize("scoring,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("offsets", [None, [0, 2, 2, 5], [1, 4]])
def test_route_backward_is_the_derivative(scoring, renorm, offsets):
    rng = np.random.default_rng(4)
    T, E, k = 6, 5, 3
    l, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[0, 1] = ids[0, 0]          # the same expert twice
    ids[1, 2] = -1                 # dropped assignments
    ids[2, 0] = E
    _, counts, _ = layer.balance_loss(l, ids, k, scoring, 0.3, 0.2, offsets)
    d, mag = layer.route_backward(l, ids, k, scoring, renorm, 1.7, dw, counts, 0.3, 0.2, offsets)
    inside = np.zeros(T, dtype=bool)
    for a, b in layer._spans(T, offsets):
        inside[a:b] = True

    def f(v):
        loss = layer.balance_loss(v, ids, k, scoring, 0.3, 0.2, offsets)[0][0]
        return loss + (layer.route_weights(v, ids, scoring, renorm, 1.7) * dw)[inside].sum()

    _close(d, _differences(f, l))
    assert (np.abs(d) <= mag * (1 + 1e-12)).all() and (d[~inside] == 0).all()


def test_combine_backward_is_the_derivative():
    rng = np.random.default_rng(5)
    T, k, H = 3, 2, 4
    pos = rng.permutation(T * k)
    pos[3] = -1
    eo, w, dy = rng.standard_normal((T * k, H)), rng.standard_normal((T, k)), rng.standard_normal((T, H))

    def loss(w, eo):
        return sum(w[t, j] * (eo[pos[t * k + j]] @ dy[t]) for t in range(T) for j in range(k) if pos[t * k + j] >= 0)

    dw, _, rows = layer.combine_backward(dy, eo, pos, w)
    _close(dw, _differences(lambda v: loss(v, eo), w))
    deo = _differences(lambda v: loss(w, v), eo)
    full = np.zeros_like(eo)
    for r, v in rows.items():
        full[r] = v
    _close(full, deo)
