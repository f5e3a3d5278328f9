"""Edges of the operators of a model's dense layers on the GPU: rows whose first column is far from the others and rows
across the whole range in the layer norm's backward pass, activations of every bf16 value, adapters that are not finite.

Tolerances as in test_gpu_layer.py: u = 2^-24 is half a float32 step, 2^-8 half a bf16 step."""
import numpy as np
import pytest
import torch

from oracle import dense as OD, layer as OL
from test_gpu_layer import DEV, M, TINY, U, UB, bf16, f32, host, rng, within

pytestmark = pytest.mark.gpu


# ---- layer norm, backward -----------------------------------------------------------------
def _norm_gradients(h, hf, key):
    """The backward pass of h against the oracle, with the bounds of test_add_layernorm_backward: dx's terms pass at
    most 10 roundings, xhat is formed in double and rounded once, and a column's sums have one chain."""
    T, H = hf.shape
    dy, dyf = bf16(rng(51, T, H, key).standard_normal((T, H)))
    w, wf = f32(1 + 0.1 * rng(52, H, key).standard_normal(H))
    out = M.moe_add_layernorm_backward(dy, h, w, 1e-5)
    dx, dw, db, mag, dwmag, dbmag = OD.layernorm_backward(dyf, hf, wf, 1e-5)
    parts = M.binding.lib().moe_add_layernorm_backward_workspace_size(T, H) // (8 * H)
    chain = -(-T // parts) + 4 + -(-parts // 32) + 32
    within(host(out["dx"]), dx, UB * np.abs(dx) + 10 * U * (1 + UB) * mag + TINY, "dx")
    within(host(out["dweight"]), dw, (chain + 4) * U * dwmag + 1e-38, "dweight")
    within(host(out["dbias"]), db, (chain + 4) * U * dbmag + 1e-38, "dbias")


@pytest.mark.parametrize("first", [1e3, -1e4])
@pytest.mark.parametrize("H", [64, 1000, 2048, 4096, 8200, 20000])
def test_layernorm_backward_of_a_large_first_column(H, first):
    """A channel of 1000 to 10000 times the others' size: their deviations keep their digits."""
    T = 64
    h, hf = bf16(rng(50, H).standard_normal((T, H)) + np.where(np.arange(H) == 0, first, 0.0))
    _norm_gradients(h, hf, 1)


@pytest.mark.parametrize("H", [64, 1000, 2048, 4096, 8200, 20000])
def test_layernorm_backward_across_the_range(H):
    """Both signs near bf16's largest value, 3.39e38: differences of two values leave float32."""
    g = rng(53, H)
    v = g.uniform(-3.3e38, 3.3e38, (5, H))
    v[0] = 3e38 * (-1.0) ** np.arange(H)
    v[1] = 3e38
    v[1, 0] = -3e38
    v[2] = g.standard_normal(H)
    v[2, 0] = 3e38
    v[3] = g.standard_normal(H)
    h, hf = bf16(v)
    _norm_gradients(h, hf, 2)
    one = M.moe_add_layernorm_backward(h[3:4], h[3:4], torch.ones(H, device=DEV), 1e-5)
    assert all(torch.isfinite(t).all() for t in one.values())


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("H", [64, 1000, 4096, 20000])
def test_norm_backward_of_the_smallest_rows(norm, H):
    """Values at bf16's smallest steps with eps = 0, whose 1 / sqrt is beyond float32: gradients that bf16 holds are the
    formula's, and 0 where dy is 0."""
    g = rng(56, H)
    v = g.integers(-3, 4, (5, H)) * TINY
    v[4] = g.standard_normal(H) * 1e-37
    h, hf = bf16(v)
    dy, dyf = bf16(g.standard_normal((5, H)) * np.array([1e-3, 0, 1e-20, 1, 1])[:, None])
    w, wf = f32(1 + 0.1 * g.standard_normal(H))
    if norm == "layer":
        out = M.moe_add_layernorm_backward(dy, h, w, 0.0)
        dx, _, _, mag, _, _ = OD.layernorm_backward(dyf, hf, wf, 0.0)
        tol = 10 * U * (1 + UB) * mag
    else:
        out = M.moe_add_rmsnorm_backward(dy, h, w, 0.0)
        dx, _, mag, _ = OL.rmsnorm_backward(dyf, hf, wf, 0.0)
        tol = 64 * U * (1 + UB) * mag          # (the bound of test_add_rmsnorm_backward)
    got = host(out["dx"])
    assert (got[1] == 0).all() and np.abs(dx[0]).max() > 1e35
    fits = np.abs(dx) < 3.3e38
    within(got[fits], dx[fits], (UB * np.abs(dx) + tol + TINY)[fits], "dx")
    over = np.abs(dx) > 3.5e38
    assert over[3].any() and np.array_equal(got[over], np.sign(dx[over]) * np.inf)
    assert all(torch.isfinite(out[n]).all() for n in out if n != "dx")


# ---- gated block, backward ----------------------------------------------------------------
def test_gated_backward_silu_of_every_value():
    """One row with dh = u = 1, so dbias is silu' and silu themselves in float32, for every finite bf16 value."""
    K, I = 128, 1 << 16
    bits = np.arange(I, dtype=np.uint32) << 16
    with np.errstate(invalid="ignore"):
        v = bits.view(np.float32).astype(np.float64)
    v[~np.isfinite(v)] = 0.0
    q = torch.zeros(K, 2 * I, dtype=torch.uint8, device=DEV)
    w = M.LinearWeights.from_logical(q, torch.full((1, 2 * I // 128), 127, dtype=torch.uint8, device=DEV), M.QUANT_SCHEMES["fp8"])
    gu, _ = bf16(np.concatenate([v, np.ones(I)])[None])
    dh, _ = bf16(np.ones((1, I)))
    out = host(M.moe_gated_linear_backward(dh, gu, w, activation="silu", want_dx=False, want_dbias=True)["dbias"])
    act, (slope, _) = OD.activation(v, "silu"), OD.activation_slope(v, "silu")
    with np.errstate(over="ignore"):
        p, n = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
    # p within 5 u and 1 - p within 6 u; v p one rounding more, then p + (v p)(1 - p) with one.  Where p is below 2^-126 it
    # may be 0: v p is below 2^-119 there
    far = 2.0 ** -118
    within(out[I:], act, 6.1 * U * np.abs(act) + far, "silu")
    within(out[:I], slope, 5.1 * U * p + 12.1 * U * np.abs(act) * n + U * np.abs(slope) + far, "slope")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_backward_of_large_factors(act):
    """dh u beyond float32 where the slope brings the product back: finite, and the formula's value."""
    T, K, I = 70, 128, 96
    g = rng(55)
    gate = g.uniform(-9.0, -3.0, (T, I))      # slopes of 1e-1 to 1e-17
    size = 10.0 ** g.uniform(10.0, 28.0, (T, I))
    u = size * g.choice([-1.0, 1.0], (T, I))
    gu, guf = bf16(np.concatenate([gate, u], 1))
    dh, dhf = bf16(10.0 ** g.uniform(38.0, 41.0, (T, I)) / size)
    w = M.LinearWeights.from_logical(torch.zeros(K, 2 * I, dtype=torch.uint8, device=DEV),
                                     torch.full((1, 2), 127, dtype=torch.uint8, device=DEV), M.QUANT_SCHEMES["fp8"])
    d = host(M.moe_gated_linear_backward(dh, gu, w, activation=act, want_dx=False)["dgu"])
    v, mag = OD.gated_backward(dhf, guf[:, :I], guf[:, I:], act)
    x = np.abs(guf[:, :I])
    rel = 2 * (3 * np.maximum(x, x * x) + 40) * U      # (the bound of test_gated_linear_backward)
    tol = np.concatenate([rel, rel], 1) * mag
    fits = np.abs(v) < 3.3e38
    assert (np.abs(dhf * guf[:, I:])[fits[:, :I]] > 3.5e38).sum() > 1000
    within(d[fits], v[fits], (tol + UB * (np.abs(v) + tol) + TINY)[fits], "dgu")
    over = np.abs(v) > 3.5e38
    assert np.array_equal(d[over], np.sign(v[over]) * np.inf)


# ---- adapters -----------------------------------------------------------------------------
@pytest.mark.parametrize("T,seqs,dt", [(40, None, torch.bfloat16), (70, [0, 0, 33, 70], torch.float32), (2300, [0, 900, 900, 2300], torch.bfloat16)])
def test_lora_of_an_infinite_b(T, seqs, dt):
    """An infinity and a NaN of b reach their own column in the rows of their own adapter, and nothing else."""
    K, N, R, n = 264, 208, 40, 3
    g = rng(54, T)
    x, r = bf16(g.standard_normal((T, K)))[0], torch.from_numpy(g.standard_normal((T, N))).to(DEV, dt)
    a, b = bf16(g.standard_normal((n, R, K)) / 16)[0], bf16(g.standard_normal((n, N, R)) / 8)[0]
    ids = torch.from_numpy(g.integers(0, n, T) if seqs is None else np.array([1, 0, 2])).to(DEV, torch.int32)
    off = None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device=DEV)
    want = M.moe_lora(x, M.LoraWeights(a, b), ids, off, r, dt)
    bad = b.clone()
    bad[1, 7, 3], bad[2, N - 1, R - 1] = float("inf"), float("nan")
    got = M.moe_lora(x, M.LoraWeights(a, bad), ids, off, r, dt)
    row = ids.cpu().numpy() if seqs is None else np.repeat([1, 0, 2], np.diff(seqs))
    hit = np.zeros((T, N), bool)
    hit[row == 1, 7], hit[row == 2, N - 1] = True, True
    assert np.array_equal(~np.isfinite(host(got)), hit)
    assert np.array_equal(host(got)[~hit], host(want)[~hit])
