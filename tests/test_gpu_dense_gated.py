"""The gated feed-forward block on the GPU against the float64 oracle (oracle/dense.py); tolerances as in
test_gpu_layer.py.  Its products are the linear layer's: whole-number operands make their sums exact."""
import numpy as np
import pytest
import torch

from oracle import dense as OD
from test_gpu_guards import Arena
from test_gpu_layer import TINY, U, UB, _linear_inputs, bf16, f32, host, rng, within

pytestmark = pytest.mark.gpu

M = pytest.importorskip("mixture_experts_fp8_amd")
B = M.binding
DEV = "cuda"

CASES = [  # T, K, I, scheme, act, bias: every variant of the launch rule, with ragged rows and columns
    (1, 128, 32, "fp8", "none", False), (1, 7168, 128, "fp8", "silu", False), (1, 1152, 96, "mxfp8", "gelu", True),
    (3, 256, 64, "mxfp8", "silu", True), (15, 384, 224, "fp8", "relu", True), (32, 2816, 768, "mxfp8", "gelu_tanh", True),
    (16, 256, 4128, "fp8", "silu", True), (8, 128, 8224, "mxfp8", "gelu", True), (3, 384, 8224, "fp8", "none", True),
    (33, 128, 2080, "mxfp8", "relu", True), (64, 896, 160, "fp8", "gelu", False), (100, 640, 1184, "fp8", "silu", True),
    (64, 256, 4192, "mxfp8", "none", True), (130, 256, 2080, "fp8", "gelu_tanh", True), (200, 384, 1824, "mxfp8", "silu", True),
    (257, 128, 992, "fp8", "none", True), (700, 128, 2080, "fp8", "gelu", True), (1000, 384, 2016, "mxfp8", "silu", True),
    (1750, 1664, 2144, "fp8", "gelu_tanh", True), (1900, 384, 1440, "fp8", "none", True), (1900, 512, 1440, "mxfp8", "silu", False),
    (2047, 768, 1152, "fp8", "gelu", True), (2900, 256, 3104, "mxfp8", "none", True), (3000, 128, 3104, "fp8", "relu", True),
    (2850, 640, 3104, "fp8", "silu", False), (900, 15232, 3616, "fp8", "silu", True), (900, 15104, 3616, "fp8", "none", False),
    (40, 32768, 32, "fp8", "silu", False), (60, 128, 8224, "fp8", "silu", True),
]


def _operands(T, K, I, scheme, act, bias, key=1):
    xq, xs, w, xv, wv = _linear_inputs(T, K, 2 * I, scheme, key)
    if act not in ("none", "relu"):     # activations near their bend: sums of order 1
        xs -= 12
        xv = xv * 2.0 ** -12
    w.bias, bf = f32(rng(31, T, K, I).standard_normal(2 * I)) if bias else (None, None)
    return xq, xs, w, xv, wv, bf


@pytest.mark.parametrize("T,K,I,scheme,act,bias", CASES)
def test_gated_linear(T, K, I, scheme, act, bias):
    print("gated", T, K, I, scheme, act, bias, flush=True)
    xq, xs, w, xv, wv, bf = _operands(T, K, I, scheme, act, bias)
    out = M.moe_gated_linear(xq, xs, w, act, want_gu=True)
    h, g, u = OD.gated(xv, wv, bf, act)
    gu = np.concatenate([g, u], 1)
    eb = U if bias else 0.0            # the bias's addition
    within(host(out["gu"]), gu, UB * np.abs(gu) * (1 + eb) + eb * np.abs(gu) + TINY, "gu")
    # the activation is a few u of its value off, and moves by at most 2 times what its argument does; the
    # product rounds once
    a = np.abs(OD.activation(g, act))
    tol = np.abs(u) * (16 * U * (np.abs(g) + a)) + 4 * U * np.abs(h) if bias or act not in ("none", "relu") else U * np.abs(h)
    within(host(out["h"]), h, tol + UB * (np.abs(h) + tol) + TINY, "h")
    # the same bits without gu, and again
    again = M.moe_gated_linear(xq, xs, w, act)
    assert again["gu"] is None and torch.equal(again["h"], out["h"])


@pytest.mark.parametrize("scheme", ["fp8", "mxfp8"])
def test_gated_linear_is_two_linear_layers(scheme):
    """gu is what moe_linear gives for the same columns; rows do not depend on the batch."""
    T, K, I = 700, 512, 640
    xq, xs, w, _, _ = _linear_inputs(T, K, 2 * I, scheme, 2)
    out = M.moe_gated_linear(xq, xs, w, "silu", want_gu=True)
    assert torch.equal(out["gu"], M.moe_linear(xq, xs, w))
    for rows in (slice(0, 1), slice(5, 70), slice(100, 612)):
        part = M.moe_gated_linear(xq[rows].contiguous(), xs[rows].contiguous(), w, "silu")
        assert torch.equal(part["h"], out["h"][rows])


@pytest.mark.parametrize("T,K,I,scheme", [(3, 256, 96, "fp8"), (70, 384, 224, "mxfp8"), (300, 256, 1056, "fp8"),
                                          (1500, 256, 2080, "fp8"), (2900, 256, 3104, "mxfp8")])
def test_gated_linear_stays_inside_its_buffers(T, K, I, scheme):
    xq, xs, w, _, _ = _linear_inputs(T, K, 2 * I, scheme, 3)
    want = M.moe_gated_linear(xq, xs, w, "silu", want_gu=True)
    a = Arena([2 * T * I, 4 * T * I])
    call = M.MoeGatedLinear(xq, xs, w, "silu", want_gu=True)
    call.args.h, call.args.gu = a.ptr(0), a.ptr(1)
    call()
    a.assert_guards(f"gated {T} {K} {I}")
    assert torch.equal(a.view(0, torch.bfloat16, (T, I)), want["h"])
    assert torch.equal(a.view(1, torch.bfloat16, (T, 2 * I)), want["gu"])


# ---- backward ----------------------------------------------------------------------------
BWD = [  # T, K, I, scheme, act, bias: each variant of both products, ragged rows and columns
    (1, 128, 32, "fp8", "silu", True), (3, 256, 96, "mxfp8", "gelu", True), (64, 384, 32, "fp8", "relu", False),
    (65, 128, 160, "mxfp8", "gelu_tanh", True), (100, 2816, 224, "fp8", "silu", True), (200, 384, 800, "mxfp8", "none", True),
    (300, 1152, 64, "fp8", "gelu", False), (700, 2048, 288, "mxfp8", "silu", True), (1000, 640, 1056, "fp8", "gelu_tanh", True),
    (1900, 2176, 96, "fp8", "silu", False), (2047, 768, 1152, "fp8", "gelu", True), (130, 4096, 1184, "mxfp8", "relu", True),
    (2500, 4224, 128, "fp8", "none", False), (300, 2560, 2336, "fp8", "silu", True), (4100, 4096, 64, "mxfp8", "silu", True),
    (17000, 128, 32, "fp8", "gelu", True), (5, 32768, 32, "mxfp8", "silu", True), (70, 128, 16352, "fp8", "gelu_tanh", True),
]


def _bwd_inputs(T, K, I, scheme, key=1, whole=False):
    xq, xs, w, xv, wv = _linear_inputs(T, K, 2 * I, scheme, 7 + key)
    g = rng(41, T, K, I, key)
    draw = (lambda *s: g.integers(-3, 4, s).astype(np.float64)) if whole else (lambda *s: g.standard_normal(s))
    gu, guf = bf16(draw(T, 2 * I) * (1 if whole else 2))
    dh, dhf = bf16(draw(T, I))
    return xq, xs, w, xv, wv, gu, guf, dh, dhf


@pytest.mark.parametrize("T,K,I,scheme,act,bias", BWD)
def test_gated_linear_backward(T, K, I, scheme, act, bias):
    print("gated backward", T, K, I, scheme, act, bias, flush=True)
    xq, xs, w, xv, wv, gu, guf, dh, dhf = _bwd_inputs(T, K, I, scheme)
    out = M.moe_gated_linear_backward(dh, gu, w, xq, xs, act, want_dbias=bias)
    v, mag = OD.gated_backward(dhf, guf[:, :I], guf[:, I:], act)
    # a few u of each term (the activations' bound at |v| below 20: (3 x + 32) u, on the slope's terms twice)
    x = np.abs(guf[:, :I])
    rel = 2 * (3 * np.maximum(x, x * x) + 40) * U
    # A logistic p below 2^-126, float32's smallest normal number, may be formed as 0, where act' is p (1 + x q s) with
    # |x s| <= 20 * 1.6 (1 + 0.14 * 400) < 2^11 and act is x p: off by at most 2^-115 of what they multiply.
    far = 2.0 ** -115 * np.abs(dhf)
    tol = np.concatenate([rel, rel], 1) * mag + np.concatenate([far * np.abs(guf[:, I:]), far], 1)
    d = host(out["dgu"])
    within(d, v, tol + UB * (np.abs(v) + tol) + TINY, "dgu")
    # the products are those of the dgu that came out: sums of n terms in any order
    def product(got, a, b, rounding, what):
        ref, m = a @ b, np.abs(a) @ np.abs(b)
        t = (a.shape[1] + 8) * U * m
        within(host(got), ref, t + rounding * (np.abs(ref) + t) + (TINY if rounding else 0), what)
    product(out["dx"], d, wv.T, UB, "dx")
    product(out["dw"], xv.T, d, 0, "dw")
    def bias_sums(got):
        within(host(got), v.sum(0), tol.sum(0) + (T / 256 + 64) * U * mag.sum(0) + 1e-38, "dbias")
    if bias:
        bias_sums(out["dbias"])
    else:
        assert out["dbias"] is None
    # the same bits again, and over gu
    over = gu.clone()
    again = M.MoeGatedLinearBackward(dh, over, w, xq, xs, act, want_dbias=bias, dgu=over)()
    assert torch.equal(over, out["dgu"])
    assert all(torch.equal(again[n], out[n]) for n in out if out[n] is not None)
    # parts of it (the order of the sums is chosen for the outputs that are asked for), weights' gradients in bf16
    half = M.moe_gated_linear_backward(dh, gu, w, xq, xs, act, want_dx=False, want_dbias=False, dw_dtype=torch.bfloat16)
    assert half["dx"] is half["dbias"] is None and torch.equal(half["dgu"], out["dgu"])
    product(half["dw"], xv.T, d, UB, "dw in bf16")
    rest = M.moe_gated_linear_backward(dh, gu, w, activation=act, want_dbias=bias)
    assert rest["dw"] is None and torch.equal(rest["dgu"], out["dgu"])
    product(rest["dx"], d, wv.T, UB, "dx alone")
    only = M.moe_gated_linear_backward(dh, gu, w, activation=act, want_dx=False, want_dbias=bias)
    assert torch.equal(only["dgu"], out["dgu"]) and only["dx"] is only["dw"] is None
    if bias:
        assert torch.equal(rest["dbias"], out["dbias"])
        bias_sums(only["dbias"])


@pytest.mark.parametrize("T,K,I,scheme", [(5, 128, 32, "fp8"), (77, 384, 96, "mxfp8"), (300, 256, 416, "fp8"), (1100, 512, 96, "mxfp8")])
def test_gated_linear_backward_exact(T, K, I, scheme):
    """Whole numbers without activation: dgu is below 10, every product below 2^7 10 and every sum below 2^24, so
    all gradients are exact."""
    xq, xs, w, xv, wv, gu, guf, dh, dhf = _bwd_inputs(T, K, I, scheme, 2, whole=True)
    out = M.moe_gated_linear_backward(dh, gu, w, xq, xs, "none", want_dbias=True)
    d = np.concatenate([dhf * guf[:, I:], dhf * guf[:, :I]], 1)
    assert np.array_equal(host(out["dgu"]), d)
    assert np.array_equal(host(out["dw"]), xv.T @ d) and np.array_equal(host(out["dbias"]), d.sum(0))
    assert torch.equal(out["dx"].cpu(), torch.from_numpy(d @ wv.T).to(torch.bfloat16))


def test_gated_linear_backward_extreme_sums():
    """Sums at the ends of bf16's range, zeros of both signs, infinities and NaN stay in their own rows."""
    T, K, I = 9, 128, 32
    xq, xs, w, xv, wv, gu, guf, dh, dhf = _bwd_inputs(T, K, I, "fp8", 3)
    big = [0.0, -0.0, 1e-40, -1e-40, 100.0, -100.0, 1e20, -1e20, 3e38, -3e38]
    for act in ("relu", "silu", "gelu", "gelu_tanh", "none"):
        g2 = gu.clone()
        g2[1, :len(big)] = torch.tensor(big).to(torch.bfloat16)
        g2[1, I:] = 1.0
        g2[2, 3], g2[3, I + 4] = float("nan"), float("inf")
        out = M.moe_gated_linear_backward(dh, g2, w, xq, xs, act)
        d = host(out["dgu"])
        got = np.concatenate([d[1, :len(big)], d[1, I:I + len(big)]])
        assert np.isfinite(got[:len(big)]).all(), act
        # far out every activation is 0 or the identity, with slope 0 or 1; near 0 the slope is that of 0
        slope0 = {"relu": 0.0, "silu": 0.5, "gelu": 0.5, "gelu_tanh": 0.5, "none": 1.0}[act]
        for i, b in enumerate(big):
            s = (1.0 if b > 1 else 0.0 if b < -1 else slope0) if act != "none" else 1.0
            if act == "relu" and b == 1e-40:
                s = 1.0
            assert abs(got[i] - dhf[1, i] * s) <= UB * abs(dhf[1, i]) + 1e-30, (act, b)
        clean = [0, 4, 5, 6, 7, 8]
        ref = M.moe_gated_linear_backward(dh, gu, w, xq, xs, act)
        assert torch.equal(out["dgu"][clean], ref["dgu"][clean]) and torch.equal(out["dx"][clean], ref["dx"][clean])
        assert np.isnan(d[2, I + 3]) and not np.isfinite(d[3, 4]), act


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "none"])
def test_gated_linear_backward_against_differences(act):
    T, K, I = 4, 128, 32
    xq, xs, w, xv, wv, _, _, dh, dhf = _bwd_inputs(T, K, I, "fp8", 4)
    xv, wv = xv / 64, wv / 64       # sums of order 1
    xs -= 6
    w.w_scale -= 6
    fwd = M.moe_gated_linear(xq, xs, w, act, want_gu=True)
    out = M.moe_gated_linear_backward(dh, fwd["gu"], w, xq, xs, act)
    step = 1e-6
    def f(x_, w_):
        return (OD.gated(x_, w_, None, act)[0] * dhf).sum()
    g = rng(42)
    # gu is rounded to bf16 (2^-8 of it) before the gradient is taken, dgu after: on the sums' terms
    gu = xv @ wv
    _, smag = OD.gated_backward(np.abs(dhf), gu[:, :I], gu[:, I:], act)
    size = np.abs(smag) + np.abs(np.concatenate([dhf * (1 + np.abs(gu[:, I:])), dhf * (1 + np.abs(gu[:, :I]))], 1)) * \
        (1 + np.abs(gu[:, :I]).repeat(2, 1).reshape(T, 2 * I))
    for _ in range(12):
        i, k, n = g.integers(T), g.integers(K), g.integers(2 * I)
        hi, lo = xv.copy(), xv.copy()
        hi[i, k] += step
        lo[i, k] -= step
        num = (f(hi, wv) - f(lo, wv)) / (2 * step)
        assert abs(host(out["dx"])[i, k] - num) <= 4 * UB * (size[i] @ np.abs(wv[k])) + 1e-4
        hi, lo = wv.copy(), wv.copy()
        hi[k, n] += step
        lo[k, n] -= step
        num = (f(xv, hi) - f(xv, lo)) / (2 * step)
        assert abs(host(out["dw"])[k, n] - num) <= 4 * UB * (np.abs(xv[:, k]) @ size[:, n]) + 1e-4


@pytest.mark.parametrize("T,K,I,scheme", [(3, 256, 96, "fp8"), (70, 384, 224, "mxfp8"), (300, 256, 1056, "fp8"), (1500, 2304, 352, "fp8")])
def test_gated_linear_backward_stays_inside_its_buffers(T, K, I, scheme):
    xq, xs, w, _, _, gu, _, dh, _ = _bwd_inputs(T, K, I, scheme, 5)
    want = M.moe_gated_linear_backward(dh, gu, w, xq, xs, "silu", want_dbias=True)
    n = B.lib().moe_gated_linear_backward_workspace_size(T, K, I, 1, 1, 1)
    a = Arena([4 * T * I, 2 * T * K, 8 * K * I, 8 * I, n])
    call = M.MoeGatedLinearBackward(dh, gu, w, xq, xs, "silu", want_dbias=True)
    call.args.dgu, call.args.dx, call.args.dw, call.args.dbias, call.args.workspace = (a.ptr(i) for i in range(5))
    call.args.workspace_bytes = n
    call()
    a.assert_guards(f"gated backward {T} {K} {I}")
    for i, (name, t) in enumerate((("dgu", torch.bfloat16), ("dx", torch.bfloat16), ("dw", torch.float32), ("dbias", torch.float32))):
        assert torch.equal(a.view(i, t, want[name].shape), want[name]), name
