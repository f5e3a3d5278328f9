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
