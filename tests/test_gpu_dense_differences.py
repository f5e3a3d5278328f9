"""Gradients of the dense layers' operators on the GPU against central differences of the oracle's forward functions.

The values that a forward pass leaves rounded (y, the sums) enter the differences as they are: the oracle's
function is shifted by each rounding, held constant, so the gradient is taken where the kernels take it.  What remains
are the roundings of dgu and of the block's dx to bf16, carried through the following product entry by entry, each at
its worst sign.  The last check of each test shows that these bounds notice a missing term.

u = 2^-24 is half a float32 step, 2^-8 half a bf16 step (relative)."""
import numpy as np
import pytest
import torch

from oracle import dense as OD
from test_gpu_layer import DEV, M, U, UB, _linear_inputs, bf16, f32, host, rng, within

pytestmark = pytest.mark.gpu

# Central differences with this step: step^2 / 6 of a third derivative, below 1e-8 of the gradients' scale here, and
# 2^-53 of the loss over the step, below 1e-9 of it.
STEP, DIFF = 1e-5, 1e-7


def _differences(f, x, step=STEP):
    """Differences of f by every entry of x.  f gives a vector, of which entry (i, j) of x touches entry i only, or, for
    x of one row, entry j only."""
    d = np.zeros_like(x)
    if len(x) == 1:
        d[0] = (f(x + step) - f(x - step)) / (2 * step)
        return d
    for j in range(x.shape[1]):
        e = np.zeros_like(x)
        e[:, j] = step
        d[:, j] = (f(x + e) - f(x - e)) / (2 * step)
    return d


def _noticed(mutant, num, tol, share, what):
    """At least this share of a wrong gradient's entries lies beyond the tolerance."""
    got = np.mean(np.abs(mutant - num) > tol)
    assert got >= share, f"{what}: only {got:.3f} of the entries"


def _terms(g, u, dh, act):
    """dgu, and dgu without one of the terms that it is made of."""
    d, _ = OD.gated_backward(dh, g, u, act)
    half = g.shape[1]
    gate, up = d.copy(), d.copy()
    gate[:, :half], up[:, half:] = 0, 0
    wrong = {"no gate half": gate, "no up half": up, "swapped halves": np.roll(d, half, axis=1)}
    if act not in ("none", "relu"):
        p = OD.activation(g, act) / g
        wrong["slope without its second term"] = np.concatenate([dh * u * p, d[:, half:]], 1)
        wrong["slope without its first term"] = np.concatenate([d[:, :half] - dh * u * p, d[:, half:]], 1)
    return d, wrong


@pytest.mark.parametrize("scheme", ["fp8", "mxfp8"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "none"])
def test_gated_linear_gradients(act, scheme):
    T, K, I = 13, 128, 32
    xq, xs, w, xv, wv = _linear_inputs(T, K, 2 * I, scheme, 61)
    xv, wv = xv / 32, wv / 16            # sums of order 1
    xs -= 5
    w.w_scale -= 4
    w.bias, bf = f32(0.5 * rng(62).standard_normal(2 * I))
    dh, dhf = bf16(rng(63).standard_normal((T, I)))
    fwd = M.moe_gated_linear(xq, xs, w, act, want_gu=True)
    gu = host(fwd["gu"])
    off = gu - (xv @ wv + bf)            # the sums' rounding
    assert 0.5 < np.sqrt((gu * gu).mean()) < 2
    out = M.moe_gated_linear_backward(dh, fwd["gu"], w, xq, xs, act)
    g, u = gu[:, :I], gu[:, I:]

    def loss(x_, w_, b_):                # [T, I]: row t depends on row t of x, column j on columns j of g and u
        v = x_ @ w_ + b_ + off
        return OD.activation(v[:, :I], act) * v[:, I:] * dhf
    d, wrong = _terms(g, u, dhf, act)
    # dgu: the bound of test_gated_linear_backward (a few u of each term), then its rounding
    _, mag = OD.gated_backward(dhf, g, u, act)
    x = np.abs(np.concatenate([g, g], 1))
    err = 2 * (3 * np.maximum(x, x * x) + 40) * U * mag
    ed = err + UB * (np.abs(d) + err)
    products = {   # name: (differences, bound, the product of a dgu)
        "dx": (_differences(lambda x_: loss(x_, wv, bf).sum(1), xv), ed @ np.abs(wv).T, lambda v: v @ wv.T, UB),
        "dw": (np.zeros((K, 2 * I)), np.abs(xv).T @ ed, lambda v: xv.T @ v, 0.0),
        "dbias": (np.zeros((1, 2 * I)), err.sum(0)[None], lambda v: v.sum(0)[None], 0.0)}
    for half in range(2):                # a step in all columns of one half: column j of the loss is column j's
        cols = slice(half * I, half * I + I)
        for k in range(K):
            def by_row(r):
                w_ = wv.copy()
                w_[k, cols] = r[0]
                return loss(xv, w_, bf).sum(0)
            products["dw"][0][k, cols] = _differences(by_row, wv[k:k + 1, cols])[0]
        def by_bias(r):
            b_ = bf.copy()
            b_[cols] = r[0]
            return loss(xv, wv, b_).sum(0)
        products["dbias"][0][0, cols] = _differences(by_bias, bf[None, cols])[0]
    for name, (num, carried, product, rounding) in products.items():
        # sums of n terms in float32, in any order, and the result's own rounding
        n = {"dx": 2 * I, "dw": T, "dbias": T}[name]
        ref = {"dx": np.abs(d) @ np.abs(wv).T, "dw": np.abs(xv).T @ np.abs(d), "dbias": np.abs(d).sum(0)[None]}[name]
        tol = carried + (n + 8) * U * ref
        tol += rounding * (np.abs(num) + tol) + DIFF * (1 + ref)
        got = host(out[name]).reshape(num.shape)
        within(got, num, tol, name)
        for what, v in wrong.items():
            # (a half's own columns, in dw and dbias: the others are as they should be.  The second term of a slope
            # is small where the activation is nearly straight)
            part = np.s_[:] if name == "dx" else np.s_[:, I:] if what == "no up half" else np.s_[:, :I]
            _noticed(product(v)[part], num[part], tol[part], 0.5 if what.startswith("slope") else 0.8, f"{act} {name} with {what}")


def test_norm_and_gated_gradients():
    """d/dx of sum(dh * block(norm(x))), without the quantisation between.  A pattern that x's rows and the weights' rows
    share makes the means of g and of g xhat as large as g."""
    T, H, I = 3, 128, 32
    g = rng(64)
    pattern = np.where(np.arange(H) < H // 2, 1.0, -1.0)
    x, xf = bf16(g.standard_normal((T, H)) + pattern)
    nw, nwf = f32(1 + 0.1 * g.standard_normal(H))
    nb, nbf = f32(0.1 * g.standard_normal(H))
    w = np.round(g.standard_normal((H, 2 * I)) * 2 + 2 + 2 * pattern[:, None]) / 64      # E4M3 values as they are
    lw = M.LinearWeights.from_float(torch.from_numpy(w.astype(np.float32)).to(DEV))
    dh, dhf = bf16(g.standard_normal((T, I)) + 1)
    y = M.moe_add_layernorm(x, nw, nb, 1e-5)["y"]
    off = host(y) - OD.add_layernorm(xf, None, nwf, nbf, 1e-5)[1]
    gu = torch.from_numpy((host(y) @ w).astype(np.float32)).to(torch.bfloat16)
    guf = gu.double().numpy()
    offg = guf - host(y) @ w
    b = M.moe_gated_linear_backward(dh, gu.to(DEV), lw, activation="silu")
    dx = host(M.moe_add_layernorm_backward(b["dx"], x, nw, 1e-5)["dx"])

    def loss(xx):
        v = (OD.add_layernorm(xx, None, nwf, nbf, 1e-5)[1] + off) @ w + offg
        return (OD.activation(v[:, :I], "silu") * v[:, I:] * dhf).sum(axis=1)
    num = _differences(loss, xf)
    # dgu's bound and rounding as above, through the product and its rounding, through the norm's gradient
    d, mag = OD.gated_backward(dhf, guf[:, :I], guf[:, I:], "silu")
    err = 2 * (3 * np.maximum(np.abs(guf), guf * guf) + 40) * U * mag
    ed = err + UB * (np.abs(d) + err)
    dy, ady = d @ w.T, np.abs(d) @ np.abs(w).T
    ey = ed @ np.abs(w).T + (2 * I + 8) * U * ady
    ey += UB * (np.abs(dy) + ey)
    m = xf.mean(1, keepdims=True)
    r = 1 / np.sqrt(((xf - m) ** 2).mean(1, keepdims=True) + 1e-5)
    xh, gy, eg = (xf - m) * r, dy * nwf, ey * np.abs(nwf)
    mean = lambda v: v.mean(1, keepdims=True)
    tol = r * (eg + mean(eg) + np.abs(xh) * mean(eg * np.abs(xh)))
    tol += 10 * U * r * (np.abs(gy) + mean(np.abs(gy)) + np.abs(xh) * mean(np.abs(gy * xh)))
    tol += UB * (np.abs(num) + tol) + DIFF * (1 + r * np.abs(gy))
    within(dx, num, tol, "dx")
    xterm = xh * mean(gy * xh)
    wrong = {"no mean(g)": r * (gy - xterm), "no xhat term": r * (gy - mean(gy)), "neither": r * gy,
             "no r": gy - mean(gy) - xterm}
    for what, v in wrong.items():
        _noticed(v, num, tol, 0.8, what)
