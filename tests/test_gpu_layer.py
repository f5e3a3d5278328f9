"""The operators around the expert step on the GPU against the float64 oracle (oracle/layer.py).

Tolerances.  u = 2^-24 is half a float32 step, 2^-8 half a bf16 step (relative).  A float32 sum of
n terms whose longest chain of additions has c of them is off by at most (c + 2) u times the sum
of the terms' magnitudes; each test names its chains.  Matrix-core sums follow the repository's
accumulation model (oracle.moe.ACC_ERR times the Euclidean norm of the products).
"""
import dataclasses

import numpy as np
import pytest
import torch

import harness as HN
from oracle import codec, layer as OL, moe as omoe, mx, routing as orouting
from oracle.w8a16 import bf16_rne
from test_gpu_guards import Arena

pytestmark = pytest.mark.gpu

M = pytest.importorskip("mixture_experts_fp8_amd")
B = M.binding
DEV = "cuda"
U, UB = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -133      # smallest bf16 step


def rng(*key):
    return np.random.default_rng(list(key))


def bf16(a):
    """float64 array -> bf16 GPU tensor (values rounded) and its exact values."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.to(DEV), HN.bf16_to_f64(t)


def f32(a):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.to(DEV), t.numpy().astype(np.float64)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def strided(t, pad):
    """The same matrix with rows `pad` elements further apart, NaN between them."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def within(got, want, tol, what=""):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond tolerance, worst " \
        f"{np.max(np.abs(got - want) / np.maximum(tol, 1e-300)):.3g} of it, first at {np.argwhere(bad)[0]}"


# ---- residual + RMS norm ------------------------------------------------------------------
NORM_CASES = [  # T, H, quant, residual, stride padding
    (1, 128, "fp8", True, 0), (1, 8, None, True, 0), (3, 136, None, False, 8), (5, 512, "mxfp8", True, 0),
    (7, 520, None, True, 16), (32, 2816, "fp8", True, 0), (9, 768, "w4a8", False, 0), (33, 4096, "fp8", False, 8),
    (4, 4104, None, True, 0), (6, 7168, "mxfp8", True, 8), (2, 8192, "fp8", True, 0), (3, 8224, "mxfp8", False, 0),
    (2, 16384, "fp8", True, 0), (2, 16512, "fp8", True, 0), (1, 32768, "mxfp8", True, 0), (257, 256, "fp8", True, 0),
]


def _norm_inputs(T, H, key):
    g = rng(7, T, H, key)
    x, xf = bf16(g.standard_normal((T, H)) * np.where(g.random(H) < 0.02, 20.0, 1.0))
    r, rf = bf16(g.standard_normal((T, H)))
    w, wf = f32(1 + 0.1 * g.standard_normal(H))
    return x, xf, r, rf, w, wf


def _check_codes(out, y, quant):
    """The codes are the library's own quantisation of y, and the oracle's."""
    q, s = M.moe_quant_act(y) if quant == "fp8" else M.moe_quant_act_mx(y)
    assert torch.equal(out["yq"], q) and torch.equal(out["ys"], s)
    rq, rs = (codec.quant_rows_128 if quant == "fp8" else mx.quant_rows_32)(HN.bf16_to_f64(y))
    assert np.array_equal(out["yq"].cpu().numpy(), rq) and np.array_equal(out["ys"].cpu().numpy(), rs)


@pytest.mark.parametrize("T,H,quant,residual,pad", NORM_CASES)
def test_add_rmsnorm(T, H, quant, residual, pad):
    x, xf, r, rf, w, wf = _norm_inputs(T, H, 1)
    xs, rs = (strided(x, pad), strided(r, pad)) if pad else (x, r)
    out = M.moe_add_rmsnorm(xs, w, 1e-6, residual=rs if residual else None,
                            quant=None if quant is None else M.QUANT_SCHEMES[quant])
    h, y = OL.add_rmsnorm(xf, rf if residual else None, wf, 1e-6)
    if residual:
        assert np.array_equal(host(out["h"]), h)
    else:
        assert out["h"] is None
    # y is formed in double (H additions, root and products: < 2^-30 off even at the longest rows) and
    # rounded once: the definition's bf16 value, but for values within 2^-30 of a tie
    near = np.abs(bf16_rne(y * (1 + 2.0 ** -30)) - bf16_rne(y * (1 - 2.0 ** -30))) > 0
    assert np.array_equal(host(out["y"])[~near], bf16_rne(y)[~near]) and near.mean() < 1e-4
    if quant:
        _check_codes(out, out["y"], quant)
    # outputs on request only, and in place: h over the residual, then over x
    again = M.moe_add_rmsnorm(xs, w, 1e-6, residual=rs if residual else None, want_y=False,
                              quant=None if quant is None else M.QUANT_SCHEMES[quant],
                              h=torch.empty_like(x) if quant is None else None)
    assert again["y"] is None and (quant is None or torch.equal(again["yq"], out["yq"]))
    if residual and not pad:
        for over in ("residual", "x"):
            a, b = x.clone(), r.clone()
            got = M.moe_add_rmsnorm(a, w, 1e-6, residual=b, h=b if over == "residual" else a)
            assert torch.equal(got["h"], out["h"]) and torch.equal(got["y"], out["y"])
            assert torch.equal(a if over == "residual" else b, x if over == "residual" else r)
    if not residual and not pad:
        a = x.clone()
        got = M.MoeAddRmsNorm(a, w, 1e-6, y=a)()
        assert torch.equal(got["y"], out["y"])


def test_add_rmsnorm_special_rows():
    # zero rows (0, not NaN), rows of the smallest and largest values, infinities and NaN stay in
    # their own rows; eps = 0 on a zero row gives NaN as the formula does
    H = 256
    g = rng(8)
    v = g.standard_normal((8, H))
    v[0] = 0
    v[1] *= 1e-38
    v[2] *= 1e18
    v[3, 5] = np.inf
    v[4, 7] = np.nan
    v[5, :128] = 0
    x, xf = bf16(v)
    w, wf = f32(np.ones(H))
    out = M.moe_add_rmsnorm(x, w, 1e-6, quant=M.MOE_QUANT_FP8_BLOCK128)
    y = host(out["y"])
    assert (y[0] == 0).all() and np.isnan(y[4]).all()
    assert np.isnan(y[3, 5]) and (np.delete(y[3], 5) == 0).all()     # inf * 0, x / inf
    fine = [1, 2, 5, 6, 7]
    _, ref = OL.add_rmsnorm(xf[fine], None, wf, 1e-6)
    within(y[fine], ref, np.abs(ref) * (UB + U) + TINY)
    q, s = M.moe_quant_act(out["y"])
    assert torch.equal(out["yq"], q) and torch.equal(out["ys"], s)
    assert (out["ys"][0] == 127).all() and out["ys"][5, 0] == 127
    assert np.isnan(host(M.moe_add_rmsnorm(x, w, 0.0)["y"][0:1])).all()
    # a sum past the largest bf16 value is infinite, as its rounding is
    big, _ = bf16(np.full((1, 8), 3.3e38))
    assert torch.isinf(M.moe_add_rmsnorm(big, w[:8].contiguous(), 1e-6, residual=big)["h"]).all()


NORM_BWD = [(1, 128), (1, 8), (2, 64), (5, 512), (4999, 184), (9000, 16), (3, 136), (5, 520), (40, 2816), (33, 4096), (4, 4104), (6, 7168), (2, 8224), (3, 16512),
            (1, 32768), (513, 256), (1100, 64), (1537, 1024), (7, 600), (2100, 968), (300, 16400), (290, 10000)]


@pytest.mark.parametrize("T,H", NORM_BWD)
@pytest.mark.parametrize("with_dh", [True, False])
def test_add_rmsnorm_backward(T, H, with_dh):
    x, xf, r, rf, w, wf = _norm_inputs(T, H, 2)
    dy, dyf = bf16(0.1 * rng(9, T, H).standard_normal((T, H)))
    out = M.moe_add_rmsnorm_backward(dy, x, w, 1e-5, dh=r if with_dh else None)
    dx, dw, mag, dwmag = OL.rmsnorm_backward(dyf, xf, wf, 1e-5, rf if with_dh else None)
    # row sums: chains <= 48 additions, then < 16 more roundings, on magnitudes `mag`
    within(host(out["dx"]), dx, UB * np.abs(dx) + 64 * U * (1 + UB) * mag + TINY, "dx")
    # weight gradient: a workgroup's rows in turn, then the partial rows (a 32nd of them in a chain, 32
    # chains); each term carries the row factor's < 64 u
    parts = B.lib().moe_add_rmsnorm_backward_workspace_size(T, H) // (4 * H)
    chain = -(-T // parts) + 4 + -(-parts // 32) + 32
    within(host(out["dweight"]), dw, (chain + 64) * U * dwmag + 1e-38, "dweight")
    again = M.moe_add_rmsnorm_backward(dy, x, w, 1e-5, dh=r if with_dh else None)
    assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["dweight"], out["dweight"])
    # without the weight gradient, and in place over dy and over dh
    a, b = dy.clone(), r.clone()
    only = M.MoeAddRmsNormBackward(a, x, w, 1e-5, dh=b if with_dh else None, want_dweight=False, dx=a)()
    assert only["dweight"] is None and torch.equal(a, out["dx"])
    if with_dh:
        got = M.MoeAddRmsNormBackward(dy, x, w, 1e-5, dh=b, dx=b)()
        assert torch.equal(b, out["dx"]) and torch.equal(got["dweight"], out["dweight"])


@pytest.mark.parametrize("H", [64, 1024, 2048, 9000, 20000])
def test_add_rmsnorm_backward_over_the_range(H):
    """Rows whose squares leave float32 on either side (eps 0), and rows that are infinite, NaN or zero."""
    g = rng(11, H)
    h = g.standard_normal((9, H)) * np.array([1e-36, 1e-30, 1e-20, 1, 1e20, 1e30, 1e37, 1, 1])[:, None]
    dy = g.standard_normal((9, H)) * np.array([1e-30, 1e-20, 1, 1, 1e15, 1e25, 1e30, 1, 1])[:, None]
    h, hf = bf16(h)
    dy, dyf = bf16(dy)
    w, wf = f32(1 + 0.1 * g.standard_normal(H))
    out = M.moe_add_rmsnorm_backward(dy, h, w, 0.0)
    dx, _, mag, _ = OL.rmsnorm_backward(dyf, hf, wf, 0.0)
    within(host(out["dx"]), dx, UB * np.abs(dx) + 64 * U * (1 + UB) * mag + TINY, "dx")
    for row in range(9):     # the weight gradient, row by row: exact sums of one term
        one = M.moe_add_rmsnorm_backward(dy[row:row + 1], h[row:row + 1], w, 0.0)
        assert torch.equal(one["dx"], out["dx"][row:row + 1])
        _, dw, _, dwmag = OL.rmsnorm_backward(dyf[row:row + 1], hf[row:row + 1], wf, 0.0)
        within(host(one["dweight"]), dw, 66 * U * dwmag + 1e-38, "dweight")
    hh = h.clone()
    hh[0, 3], hh[1, 5], hh[2] = float("inf"), float("nan"), 0
    got = M.moe_add_rmsnorm_backward(dy, hh, w, 1e-6, dh=dy)["dx"]
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    # a zero row: r = 1000, no xhat
    ref = 1000.0 * dyf[2] * wf + dyf[2]
    within(host(got[2]), ref, UB * np.abs(ref) + 64 * U * (1000 * np.abs(dyf[2] * wf) + np.abs(dyf[2])))
    assert torch.equal(got[3:], M.moe_add_rmsnorm_backward(dy[3:], h[3:], w, 1e-6, dh=dy[3:])["dx"])


def test_weight_gradient_at_any_float():
    """dweight is 4-byte aligned: a slice of a flat gradient buffer, also where one part is the whole sum."""
    for T, H in ((1, 4096), (3, 64), (9, 64)):
        x, _, r, _, w, _ = _norm_inputs(T, H, 3)
        want = M.moe_add_rmsnorm_backward(r, x, w, 1e-5)
        flat = torch.full((H + 8,), 7.0, device="cuda")
        call = M.MoeAddRmsNormBackward(r, x, w, 1e-5)
        call.args.dweight = flat[3:].data_ptr()
        call()
        assert torch.equal(flat[3:3 + H], want["dweight"])
        assert (flat[:3] == 7).all() and (flat[3 + H:] == 7).all()


def test_add_rmsnorm_backward_against_differences():
    g = rng(10)
    h, hf = bf16(g.standard_normal((3, 16)))
    dy, dyf = bf16(g.standard_normal((3, 16)))
    w, wf = f32(g.standard_normal(16))
    out = M.moe_add_rmsnorm_backward(dy, h, w, 1e-3)
    step = 1e-5
    num = np.zeros_like(hf)
    for i in range(3):
        for j in range(16):
            hi, lo = hf.copy(), hf.copy()
            hi[i, j] += step
            lo[i, j] -= step
            num[i, j] = ((OL.add_rmsnorm(hi, None, wf, 1e-3)[1] - OL.add_rmsnorm(lo, None, wf, 1e-3)[1]) * dyf).sum() / (2 * step)
    _, _, mag, _ = OL.rmsnorm_backward(dyf, hf, wf, 1e-3)
    # (the norm's input is perturbed unrounded: add_rmsnorm rounds only a sum)
    within(host(out["dx"]), num, UB * np.abs(num) + 64 * U * mag + 1e-7)


# ---- linear -------------------------------------------------------------------------------
# The scaled FP8 matrix instruction aligns the eight products of eight consecutive K to the largest
# of them and drops what lies below 2^-13 of its power of two (measured with single products; the
# sums of eights and the accumulator behave as float32).  So
#   * whole numbers up to 7 with scales 1 and 2 multiply to whole numbers up to 196: nothing is
#     dropped, and every sum stays below 196 * 32768 < 2^24, so float32 holds it exactly: those
#     inputs are checked with no allowance for the sum;
#   * on other inputs a sum of eight products is off by at most 7 * 2^-13 of their largest.
def _linear_inputs(T, K, N, scheme, key, whole=True):
    """Device operands and their exact values (numpy float64)."""
    g = rng(11, T, K, N, key)
    micro = scheme == "mxfp8"
    gs, nb = (32, N) if micro else (128, -(-N // 128))
    if whole:
        xq = codec.e4m3_encode(g.integers(-7, 8, (T, K)).astype(np.float64))
        q = codec.e4m3_encode(g.integers(-7, 8, (K, N)).astype(np.float64))
        xs = g.integers(127, 129, (T, K // gs)).astype(np.uint8)
        s = g.integers(127, 129, (K // gs, nb)).astype(np.uint8)
        xqd, xsd = torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV)
    else:
        x, _ = bf16(g.standard_normal((T, K)) * np.where(g.random(K) < 0.02, 12.0, 1.0))
        xqd, xsd = M.moe_quant_act_mx(x) if micro else M.moe_quant_act(x)
        xq, xs = xqd.cpu().numpy(), xsd.cpu().numpy()
        wf = 0.05 * g.standard_normal((K, N))
        q, s = mx.quant_weight_k32(wf, mx.FMT_E4M3) if micro else codec.quant_blocks_128(wf)
    xv, wv = OL.dequant_linear(xq, xs, q, s, micro)
    w = M.LinearWeights.from_logical(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), M.QUANT_SCHEMES[scheme])
    return xqd, xsd, w, xv, wv


def _linear_ref(xv, wv, bias, act, res):
    """(y, tolerance before the final rounding) for exact sums: the bias, the activation (a few u of
    its value; its argument's rounding moves it by less than the argument's) and the residual."""
    y, _ = OL.linear(xv, wv, bias, act, res)
    v = xv @ wv + (0 if bias is None else bias)
    if act in ("none", "relu") and bias is None and res is None:
        return y, np.zeros_like(y)
    return y, 16 * U * (np.abs(v) + np.abs(y) + (0 if res is None else np.abs(res)))


LINEAR_CASES = [  # T, K, N, scheme, act, bias, residual, out
    (1, 128, 16, "fp8", "none", False, False, "bf16"), (1, 7168, 256, "fp8", "none", False, True, "bf16"),
    (1, 1152, 144, "mxfp8", "gelu", True, True, "f32"), (3, 256, 128, "mxfp8", "silu", True, False, "bf16"),
    (15, 384, 400, "fp8", "relu", True, True, "bf16"), (16, 2816, 272, "mxfp8", "none", False, False, "f32"),
    (17, 640, 128, "fp8", "gelu", True, True, "f32"), (32, 2816, 2816, "mxfp8", "gelu", True, False, "bf16"),
    (33, 128, 48, "fp8", "silu", False, True, "bf16"), (63, 1024, 2048, "fp8", "none", False, False, "f32"),
    (64, 896, 304, "mxfp8", "relu", False, True, "bf16"), (65, 256, 256, "fp8", "gelu_tanh", True, True, "bf16"),
    (127, 512, 1040, "fp8", "none", True, True, "f32"), (128, 4096, 512, "mxfp8", "none", False, False, "bf16"),
    (129, 768, 2304, "fp8", "silu", True, False, "bf16"), (200, 2048, 4096, "fp8", "none", False, True, "bf16"),
    (255, 384, 640, "mxfp8", "silu", True, True, "f32"), (257, 1536, 1280, "mxfp8", "gelu", False, True, "bf16"),
    (300, 128, 128, "fp8", "none", False, False, "f32"), (513, 640, 784, "fp8", "relu", True, True, "bf16"),
    (700, 768, 1152, "mxfp8", "none", False, False, "f32"), (1025, 896, 2304, "fp8", "gelu", True, True, "f32"),
    (2047, 768, 2304, "fp8", "silu", True, False, "bf16"), (1500, 1024, 4112, "mxfp8", "silu", False, True, "bf16"),
    (2600, 1152, 2560, "fp8", "none", False, False, "f32"), (4100, 256, 2048, "fp8", "gelu_tanh", True, True, "bf16"),
    (40, 32768, 32, "fp8", "none", False, True, "bf16"), (300, 16512, 512, "mxfp8", "none", False, False, "f32"),
    # one of each variant by its number of workgroups, with one, two and an odd number of K blocks, K blocks
    # that are no multiple of four, and columns that end inside a tile
    (33, 384, 4112, "mxfp8", "none", True, True, "bf16"), (16, 128, 8208, "fp8", "silu", False, False, "bf16"),
    (1, 256, 8192, "mxfp8", "none", False, True, "f32"), (64, 256, 8336, "fp8", "relu", False, True, "bf16"),
    (257, 128, 1936, "fp8", "none", False, False, "f32"), (200, 256, 3600, "mxfp8", "none", False, True, "bf16"),
    (300, 32768, 1168, "fp8", "none", False, True, "bf16"), (700, 128, 4112, "fp8", "gelu", True, True, "f32"),
    (1000, 384, 3984, "mxfp8", "silu", True, True, "bf16"), (1800, 128, 4112, "mxfp8", "none", False, False, "f32"),
    (1750, 1664, 4240, "fp8", "gelu_tanh", True, True, "bf16"), (2900, 256, 6160, "mxfp8", "none", False, True, "bf16"),
    (2850, 640, 6160, "fp8", "none", True, False, "f32"), (3000, 128, 6160, "fp8", "relu", True, True, "bf16"),
    (1100, 512, 4112, "mxfp8", "gelu", True, True, "bf16"), (1900, 384, 2832, "fp8", "none", True, True, "f32"),
    (1900, 640, 3856, "fp8", "silu", True, False, "bf16"),
    (60, 128, 8208, "mxfp8", "none", True, True, "bf16"), (20, 640, 12304, "fp8", "gelu", False, True, "f32"),
    (130, 256, 4112, "fp8", "none", True, False, "bf16"), (3, 256, 16528, "fp8", "none", True, True, "bf16"),
    (8, 128, 16528, "mxfp8", "silu", False, False, "f32"), (20, 384, 16528, "mxfp8", "none", True, True, "bf16"),
    (10, 128, 32912, "fp8", "relu", True, False, "bf16"), (400, 384, 3600, "mxfp8", "gelu_tanh", True, True, "f32"),
    (400, 512, 3600, "fp8", "none", False, True, "bf16"), (64, 32768, 528, "mxfp8", "none", False, False, "bf16"),
    (900, 15104, 7184, "fp8", "none", False, True, "bf16"), (900, 15232, 7184, "fp8", "none", True, False, "bf16"),
]


@pytest.mark.parametrize("T,K,N,scheme,act,bias,residual,out", LINEAR_CASES)
def test_linear(T, K, N, scheme, act, bias, residual, out):
    print("linear", T, K, N, scheme, act, bias, residual, out, flush=True)
    xq, xs, w, xv, wv = _linear_inputs(T, K, N, scheme, 1)
    if act not in ("none", "relu"):     # activations near their bend: sums of order 1
        xs -= 12
        xv = xv * 2.0 ** -12
    g = rng(12, T, K, N)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    bd, bf = f32(g.standard_normal(N)) if bias else (None, None)
    rd, rf = (bf16 if out == "bf16" else f32)(g.standard_normal((T, N))) if residual else (None, None)
    w.bias = bd
    y = M.moe_linear(xq, xs, w, act, rd, dt)
    ref, tol = _linear_ref(xv, wv, bf, act, rf)
    within(host(y), ref, tol + (UB * (np.abs(ref) + tol) + TINY if out == "bf16" else 0))
    # the same bits again, with strided rows, and in place over the residual
    assert torch.equal(M.moe_linear(xq, xs, w, act, rd, dt), y)
    ys = torch.full((T, N + 8), 7.0, dtype=dt, device=DEV)
    got = M.moe_linear(xq, xs, w, act, strided(rd, 24) if residual else None, dt, y=ys[:, :N])
    assert torch.equal(got, y) and (ys[:, N:] == 7.0).all()
    if residual:
        over = rd.clone()
        assert torch.equal(M.moe_linear(xq, xs, w, act, over, dt, y=over), y)


@pytest.mark.parametrize("scheme", ["fp8", "mxfp8"])
@pytest.mark.parametrize("T,K,N", [(5, 2816, 128), (40, 1024, 256), (300, 512, 256)])
def test_linear_on_quantised_values(scheme, T, K, N):
    """Operands as the quantisers make them, with large channels: within what the instruction drops."""
    xq, xs, w, xv, wv = _linear_inputs(T, K, N, scheme, 4, whole=False)
    y = host(M.moe_linear(xq, xs, w, out_dtype=torch.float32))
    drop = np.zeros((T, N))
    for k in range(0, K, 8):
        drop += np.max(np.abs(xv[:, k:k + 8, None] * wv[None, k:k + 8]), axis=1)
    ref, mag = OL.linear(xv, wv)
    # beyond that: K / 8 additions of eights in float32 (twice u: the adder may cut instead of round)
    within(y, ref, 7 * 2.0 ** -13 * drop + (K / 8 + 32) * 2 * U * mag)
    # and such losses do not add up: their signs are those of the products, so over all outputs they
    # come to far less than their bound, 2^-13 of the products' norm (the repository's model)
    rms = np.sqrt(((xv * xv) @ (wv * wv)).mean())
    assert np.sqrt(((y - ref) ** 2).mean()) <= omoe.ACC_ERR * rms


@pytest.mark.parametrize("scheme", ["fp8", "mxfp8"])
def test_linear_rows_do_not_depend_on_the_batch(scheme):
    # every row of a batch is the same sum whatever the rows beside it hold
    xq, xs, w, _, _ = _linear_inputs(700, 512, 640, scheme, 2, whole=scheme == "fp8")
    y = M.moe_linear(xq, xs, w)
    perm = torch.randperm(700, generator=torch.Generator().manual_seed(3)).to(DEV)
    assert torch.equal(M.moe_linear(xq[perm].contiguous(), xs[perm].contiguous(), w), y[perm])


def test_linear_columns_side_by_side():
    """y and residual as column slices of one matrix, and a single row of a wider one in place."""
    w = M.LinearWeights.from_float(f32(rng(3).standard_normal((256, 64)))[0])
    x, _ = bf16(rng(4).standard_normal((20, 256)))
    xq, xs = M.moe_quant_act(x)
    wide = M.LinearWeights.from_float(torch.cat([f32(rng(3).standard_normal((256, 64)))[0], torch.zeros(256, 64, device=DEV)], 1))
    assert w.N == 64 and torch.equal(M.moe_linear(xq, xs, w), M.moe_linear(xq, xs, wide)[:, :64])
    both = torch.zeros(20, 128, dtype=torch.bfloat16, device=DEV)
    both[:, 64:] = bf16(rng(5).standard_normal((20, 64)))[0]
    want = M.moe_linear(xq, xs, w, residual=both[:, 64:].contiguous())
    keep = both[:, 64:].clone()
    got = M.moe_linear(xq, xs, w, residual=both[:, 64:], y=both[:, :64])
    assert torch.equal(got, want) and torch.equal(both[:, 64:], keep)
    with pytest.raises(M.MoeError):
        M.moe_linear(xq, xs, w, residual=both[:, 32:96], y=both[:, :64])
    one = both[3:4, 64:]
    M.moe_linear(xq[3:4], xs[3:4], w, residual=one, y=one)
    assert torch.equal(one, want[3:4]) and torch.equal(both[4:, 64:], keep[4:]) and torch.equal(both[3:4, :64], want[3:4])


def test_router_parameters_are_copied():
    p = M.route_params(8, 2)
    l, ids = torch.randn(4, 8, device=DEV), torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    call, back = M.MoeBalanceLoss(p, l, ids), M.MoeRouteBackward(p, l, ids, torch.ones(4, 2, device=DEV))
    a, b = call()["losses"].clone(), back().clone()
    p.top_k, p.num_experts = 8, 1024
    assert torch.equal(call()["losses"], a) and torch.equal(back(), b)


def test_linear_zero_rows_and_nan():
    xq, xs, w, _, _ = _linear_inputs(20, 256, 128, "fp8", 3)
    xq[3] = 0
    xq[5, 7] = 0x7F         # E4M3 NaN
    w.bias = torch.ones(128, device=DEV)
    y = host(M.moe_linear(xq, xs, w, "silu"))
    assert np.allclose(y[3], 0.7310585786300049, rtol=UB) and np.isnan(y[5]).all()
    keep = [i for i in range(20) if i not in (3, 5)]
    assert np.isfinite(y[keep]).all()


# ---- router losses and gradient --------------------------------------------------------------
ROUTER_CASES = [  # T, E, k, scoring, renorm, rsf, offsets
    (1, 1, 1, "softmax", False, 1.0, None), (1, 8, 2, "softmax", True, 1.0, None), (64, 8, 2, "softmax", True, 2.5, None),
    (37, 60, 4, "sigmoid", True, 2.5, [0, 11, 11, 30]), (65, 64, 6, "softmax", False, 1.0, [3, 3, 60, 65]),
    (200, 67, 3, "softmax", True, 1.0, [0, 200]), (130, 128, 8, "sigmoid", True, 1.0, None),
    (300, 130, 8, "softmax", False, 0.5, [0, 1, 2, 64, 65, 128, 290]), (257, 256, 8, "sigmoid", True, 2.5, [0, 100, 257]),
    (90, 260, 5, "softmax", True, 1.0, [0, 45, 90]), (70, 513, 8, "sigmoid", True, 1.0, [7, 7, 7, 63]),
    (50, 1024, 12, "softmax", False, 1.0, None), (40, 1001, 1, "softmax", True, 1.0, [0, 39]),
    (5000, 96, 4, "softmax", True, 1.0, [0, 2500, 2600, 4999]), (20000, 16, 2, "sigmoid", True, 1.0, None),
    (17, 10, 10, "softmax", True, 1.0, [0, 0, 17, 17]), (12, 8, 2, "softmax", False, 1.0, [5, 5]),
    (33, 100, 20, "softmax", True, 1.5, None), (21, 600, 70, "sigmoid", True, 1.0, [0, 20]),     # more slots than lanes
    (128, 32, 4, "softmax", False, 1.0, [0, 1, 1, 90, 128]), (129, 32, 4, "sigmoid", True, 1.0, [0, 1, 1, 90, 128]),
    (90, 16, 2, "softmax", True, 1.0, sorted([0, 90] + [(37 * i) % 91 for i in range(70)])),     # many short sequences
    (3000, 8, 1, "sigmoid", True, 1.0, sorted([0, 2990] + [(1231 * i) % 2991 for i in range(1500)])),
]
CA, CZ = 0.37, 0.011


def _router_inputs(T, E, k, key=1):
    g = rng(13, T, E, k, key)
    l, lf = f32(2.0 * g.standard_normal((T, E)) + 0.5 * g.standard_normal(E))
    ids = np.argsort(-lf, axis=1, kind="stable")[:, :k].astype(np.int32)
    dw, dwf = f32(g.standard_normal((T, k)))
    return l, lf, torch.from_numpy(np.ascontiguousarray(ids)).to(DEV), ids, dw, dwf


def _params(E, k, scoring, renorm, rsf=1.0):
    return M.route_params(E, k, scoring, renorm, routed_scaling_factor=rsf)


def _off(o):
    return None if o is None else torch.tensor(o, dtype=torch.int32, device=DEV)


def _check_router(l, lf, ids, idn, dw, dwf, k, scoring, renorm, rsf, offsets):
    E = l.shape[1]
    p = _params(E, k, scoring, renorm, rsf)
    out = M.moe_balance_loss(p, l, ids, _off(offsets), CA, CZ)
    losses, counts, mean = OL.balance_loss(lf, idn, k, scoring, CA, CZ, offsets)
    assert np.array_equal(out["counts"].cpu().numpy(), counts)
    fin = lf[np.isfinite(lf)]
    R = float(fin.max() - fin.min()) if fin.size else 0.0
    # a probability: exponent R u off, exp and division a few u, sum of E terms (chain <= 16 + 6);
    # sums over rows: a part's rows over 8 groups of lanes or more (chain <= T / 256 / 8 + 32), then at
    # most 256 parts one by one
    c_row = R + 40
    c_sum = c_row + len(lf) / 2048 + 32 + 256
    within(host(out["mean_probs"]), mean, c_sum * U * mean + 1e-37, "mean_probs")
    lse = max(1.0, np.abs(fin).max() if fin.size else 1.0)
    got = host(out["losses"])
    within(got[1:2], losses[1:2], (c_sum + 40) * U * abs(losses[1:2]) + 1e-37, "balance")
    # z: lse is off by < 40 u max(1, |lse|); its square by twice that
    n = max(1, sum(max(0, b - a) for a, b in OL._spans(len(lf), offsets)))
    within(got[2:3], losses[2:3], (2 * 40 + c_sum) * U * CZ * max(lse + np.log(E), 1.0) ** 2 + 1e-37, "z")
    within(got[0:1], losses[0:1], 2 * (c_sum + 120) * U * (abs(losses[1]) + CZ * max(lse + np.log(E), 1.0) ** 2) + 1e-37, "sum")
    d = M.moe_route_backward(p, l, ids, dw, out["counts"], _off(offsets), CA, CZ)
    ref, mag = OL.route_backward(lf, idn, k, scoring, renorm, rsf, dwf, counts, CA, CZ, offsets)
    # every term is a product of < 12 factors each off by < 40 u + R u, and a row sum; lse as above
    zmag = 2 * CZ / n * 40 * max(lse, 1.0)
    within(host(d), ref, (4 * c_row + 64) * U * mag + zmag * U + 1e-37, "dlogits")
    return out, d


@pytest.mark.parametrize("T,E,k,scoring,renorm,rsf,offsets", ROUTER_CASES)
def test_balance_loss_and_route_backward(T, E, k, scoring, renorm, rsf, offsets):
    l, lf, ids, idn, dw, dwf = _router_inputs(T, E, k)
    inside = np.zeros(T, dtype=bool)
    for a, b in OL._spans(T, offsets):
        inside[a:b] = True
    if not inside.all():    # what lies outside the sequences is not read
        l[torch.from_numpy(~inside).to(DEV)] = float("nan")
        ids[torch.from_numpy(~inside).to(DEV)] = 1 << 30
        dw[torch.from_numpy(~inside).to(DEV)] = float("nan")
    out, d = _check_router(l, lf, ids, idn, dw, dwf, k, scoring, renorm, rsf, offsets)
    assert (d[torch.from_numpy(~inside).to(DEV)] == 0).all()
    again, d2 = _check_router(l, lf, ids, idn, dw, dwf, k, scoring, renorm, rsf, offsets)
    assert torch.equal(d, d2) and all(torch.equal(out[n], again[n]) for n in out)
    # parts of the gradient add up: each alone, and in place over the logits
    p = _params(E, k, scoring, renorm, rsf)
    only_w = M.moe_route_backward(p, l, ids, dw, None, _off(offsets), 0.0, 0.0)
    ref, mag = OL.route_backward(lf, idn, k, scoring, renorm, rsf, dwf, None, 0.0, 0.0, offsets)
    within(host(only_w), ref, (4 * (np.ptp(lf) + 40) + 64) * U * mag + 1e-37, "weights path")
    only_z = M.moe_route_backward(p, l, None, None, None, _off(offsets), 0.0, CZ)
    ref, mag = OL.route_backward(lf, None, k, scoring, renorm, rsf, None, None, 0.0, CZ, offsets)
    within(host(only_z), ref, (4 * (np.ptp(lf) + 40) + 64) * U * mag + 2 * CZ * 40 * U * max(1.0, np.abs(lf).max()), "z path")
    over = l.clone()
    M.MoeRouteBackward(p, over, ids, dw, out["counts"], _off(offsets), CA, CZ, dlogits=over)()
    assert torch.equal(over, d)


def test_router_masked_experts_dropped_and_repeated_ids():
    T, E, k = 40, 24, 4
    l, lf, ids, idn, dw, dwf = _router_inputs(T, E, k, 2)
    for a in (lf, l):
        a[:, 20:] = -float("inf")                 # experts that no token may take
        a[7] = -float("inf")                      # a row whose mask leaves nothing
        a[9, :] = -float("inf")
        a[9, 3] = 1.5                             # one live expert
    for a in (idn, ids):
        a[2, 1] = -1                              # dropped assignments
        a[3, :] = -1
        a[4, 0] = E
        a[5, 2] = int(idn[5, 0])                  # the same expert twice, and in every slot
        a[6, :] = 11
    # more slots than a row has lanes, with repeats on both sides of that
    l2, lf2, ids2, idn2, dw2, dwf2 = _router_inputs(9, 40, 33, 9)
    for a in (idn2, ids2):
        a[0, 20] = int(idn2[0, 1])
        a[0, 32] = int(idn2[0, 1])
        a[1, :] = 7
        a[2, 16:] = -1
    for scoring, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        _check_router(l2, lf2, ids2, idn2, dw2, dwf2, 33, scoring, renorm, 0.7, None)
    for scoring, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        _, d = _check_router(l, lf, ids, idn, dw, dwf, k, scoring, renorm, 1.3, [0, 20, 38])
        assert torch.isfinite(d).all() and (d[7] == 0).all()
    # NaN and +infinity stay in their rows
    l[11, 2] = float("nan")
    l[12, 2] = float("inf")
    d = M.moe_route_backward(_params(E, k, "softmax", True), l, ids, dw, None, None, 0.0, 0.1)
    bad = torch.isnan(d).any(1).nonzero().flatten().tolist()
    assert bad == [11, 12]


def test_router_logits_at_the_ends_of_float32():
    """Masks of the type's lowest value, and logits whose exponentials or sigmoids leave float32."""
    T, E, k = 24, 16, 3
    l, lf, ids, idn, dw, dwf = _router_inputs(T, E, k, 12)
    low = float(np.finfo(np.float32).min)
    for a in (l, lf):
        a[:, 12:] = low
        a[3] = low                                # a row whose mask leaves nothing
        a[5, 2] = -low                            # one expert takes it all
        a[6] = 200.0
        a[7, :6] = -60.0
    for scoring, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        p = _params(E, k, scoring, renorm, 1.0)
        out = M.moe_balance_loss(p, l, ids, None, CA, 0.0)
        losses, counts, mean = OL.balance_loss(lf, idn, k, scoring, CA, 0.0)
        # exponents up to 400 where they are not 0 or 1: < 400 u, then as in _check_router
        within(host(out["mean_probs"]), mean, 800 * U * mean + 1e-37, "mean_probs")
        within(host(out["losses"]), losses, 900 * U * np.abs(losses) + 1e-37, "losses")
        d = M.moe_route_backward(p, l, ids, dw, out["counts"], None, CA, 0.0)
        ref, mag = OL.route_backward(lf, idn, k, scoring, renorm, 1.0, dwf, counts, CA, 0.0)
        within(host(d), ref, 4000 * U * mag + 1e-37, "dlogits")
        assert torch.isfinite(d).all() and (scoring != "sigmoid" or (d[3] == 0).all())


def test_route_backward_against_differences():
    T, E, k = 5, 12, 3
    l, lf, ids, idn, dw, dwf = _router_inputs(T, E, k, 3)
    for scoring, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        counts = OL.balance_loss(lf, idn, k, scoring, CA, CZ, [0, 2, 5])[1]

        def f(v):
            return OL.balance_loss(v, idn, k, scoring, CA, CZ, [0, 2, 5])[0][0] + \
                (OL.route_weights(v, idn, scoring, renorm, 1.7) * dwf).sum()

        num = np.zeros((T, E))
        for t in range(T):
            for e in range(E):
                hi, lo = lf.copy(), lf.copy()
                hi[t, e] += 1e-5
                lo[t, e] -= 1e-5
                num[t, e] = (f(hi) - f(lo)) / 2e-5
        d = M.moe_route_backward(_params(E, k, scoring, renorm, 1.7), l, ids, dw,
                                 torch.from_numpy(counts.astype(np.int32)).to(DEV), _off([0, 2, 5]), CA, CZ)
        # differences: 1e-10 truncation and 1e-11 rounding of values of order 1
        _, mag = OL.route_backward(lf, idn, k, scoring, renorm, 1.7, dwf, counts, CA, CZ, [0, 2, 5])
        within(host(d), num, 1e-8 + (4 * (np.ptp(lf) + 40) + 64) * U * mag + 1e-6 * CZ)


def test_single_choice_has_no_weight_gradient():
    # one expert per token, normalised over the chosen: its weight is constant
    for scoring in ("softmax", "sigmoid"):
        l, lf, ids, idn, dw, dwf = _router_inputs(500, 12, 1, 5)
        assert (M.moe_route_backward(_params(12, 1, scoring, True, 1.9), l, ids, dw, None, None, 0.0, 0.0) == 0).all()
        _check_router(l, lf, ids, idn, dw, dwf, 1, scoring, True, 1.9, None)


def test_balance_counts_are_the_routers():
    # counts of one sequence are moe_route's expert_counts
    T, E, k = 3000, 64, 6
    l = _router_inputs(T, E, k, 4)[0]
    p = _params(E, k, "softmax", True)
    r = M.moe_route(p, T, l)
    out = M.moe_balance_loss(p, l, r["topk_ids"])
    assert torch.equal(out["counts"][0], r["expert_counts"])


# ---- combine --------------------------------------------------------------------------------
COMBINE_CASES = [(1, 1, 8, "bf16"), (3, 2, 768, "f32"), (5, 8, 1024, "bf16"), (4, 9, 1032, "f32"), (2, 17, 2816, "bf16"),
                 (37, 8, 4096, "bf16"), (6, 3, 8192, "f32"), (130, 1, 264, "bf16"),
                 (256, 2, 2064, "bf16"), (257, 2, 2064, "bf16"), (9, 10, 4104, "f32"), (1030, 1, 4096, "f32"), (1024, 3, 520, "f32")]


@pytest.mark.parametrize("T,k,H,dtype", COMBINE_CASES)
def test_combine_backward(T, k, H, dtype):
    g = rng(14, T, k, H)
    mk = bf16 if dtype == "bf16" else f32
    eo, eof = mk(g.standard_normal((T * k, H)))
    dy, dyf = bf16(g.standard_normal((T, H)))
    w, wf = f32(g.random((T, k)))
    pos = g.permutation(T * k).astype(np.int32)
    if T * k > 4:
        pos[1], pos[3] = -1, T * k      # dropped assignments
    pd = torch.from_numpy(pos).to(DEV)
    fill = torch.full_like(eo, 3.0)
    out = M.moe_combine_backward(dy, eo, pd, w, d_expert_out=fill)
    dw, mag, rows = OL.combine_backward(dyf, eof, pos, wf)
    # chain: a thread's columns (<= H / 8 / 64 vectors of 8) and the tree
    within(host(out["dweights"]), dw, (H / 64 + 32) * U * mag + 1e-37, "dweights")
    got = out["d_expert_out"]
    named = torch.zeros(T * k, dtype=torch.bool, device=DEV)
    for t in range(T):
        for j in range(k):
            r = pos[t * k + j]
            if 0 <= r < T * k:      # one float32 product, rounded once more for bf16
                named[r] = True
                assert torch.equal(got[int(r)], (w[t, j] * dy[t].float()).to(eo.dtype)), (t, j)
    assert (got[~named] == 3.0).all()
    assert torch.equal(M.moe_combine_backward(dy, eo, pd, w)["dweights"], out["dweights"])
    over = eo.clone()
    both = M.moe_combine_backward(dy, over, pd, w, d_expert_out=over)
    assert torch.equal(both["dweights"], out["dweights"]) and torch.equal(over[named], got[named])
    assert torch.equal(over[~named], eo[~named])
    alone = M.moe_combine_backward(dy, eo, pd, w, d_expert_out=torch.full_like(eo, 3.0), want_dweights=False)
    assert alone["dweights"] is None and torch.equal(alone["d_expert_out"], got)


# ---- together ---------------------------------------------------------------------------------
def _layer(scheme, T=96, H=512, I=256, E=16, k=4):
    g = rng(15, T, H, E)
    quant = M.QUANT_SCHEMES[scheme]
    x, _ = bf16(g.standard_normal((T, H)))
    res, _ = bf16(g.standard_normal((T, H)))
    nw, _ = f32(1 + 0.1 * g.standard_normal(H))
    wo = M.LinearWeights.from_float(f32(0.05 * g.standard_normal((H, H)))[0], quant)
    w13, _ = f32(0.05 * g.standard_normal((E, H, 2 * I)))
    w2, _ = f32(0.05 * g.standard_normal((E, I, H)))
    if scheme == "mxfp8":
        we = M.pack_weights_mx(w13, w2, quant)
    else:
        we = M.PackedWeights.from_logical(*M.moe_quant_weight_blocks(w13), *M.moe_quant_weight_blocks(w2))
    rw, _ = f32(0.05 * g.standard_normal((H, E)))
    dy, _ = bf16(0.1 * g.standard_normal((T, H)))
    return dict(x=x, res=res, nw=nw, wo=wo, we=we, rw=rw, dy=dy, quant=quant, p=M.route_params(E, k, "softmax", True), T=T, k=k)


@pytest.mark.parametrize("scheme", ["fp8", "mxfp8"])
def test_layer_forward_and_router_gradient(scheme):
    """A layer's run of them: attention output projected onto the residual stream, normed and
    quantised once for the router and the experts, routed, combined; then back to the router."""
    c = _layer(scheme)
    p, T, k = c["p"], c["T"], c["k"]
    xq, xs = M.moe_quant_act(c["x"]) if scheme == "fp8" else M.moe_quant_act_mx(c["x"])
    att = M.moe_linear(xq, xs, c["wo"])
    n = M.moe_add_rmsnorm(att, c["nw"], residual=c["res"], quant=c["quant"])
    logits = n["y"].float() @ c["rw"]
    r = M.moe_route(p, T, logits)
    eo = M.moe_grouped_ffn(n["yq"], n["ys"], r, c["we"], k)
    y = M.moe_combine(eo, r["assign_pos"], r["topk_weights"])
    # the expert step on y itself gives the same bits: the codes are its own
    fused = M.moe_fused(p, n["y"], c["we"], router_logits=logits)
    assert torch.equal(fused, y)
    # adding the projection's residual in its epilogue rounds once where the pair rounds twice
    direct = host(M.moe_linear(xq, xs, c["wo"], residual=c["res"]))
    within(host(n["h"]), direct, 2 * UB * (np.abs(direct) + np.abs(host(att))) + TINY)
    loss = M.moe_balance_loss(p, logits, r["topk_ids"], None, CA, CZ)
    cb = M.moe_combine_backward(c["dy"], eo, r["assign_pos"], r["topk_weights"])
    d = M.moe_route_backward(p, logits, r["topk_ids"], cb["dweights"], loss["counts"], None, CA, CZ)
    dyn = (d @ c["rw"].t()).to(torch.bfloat16)
    back = M.moe_add_rmsnorm_backward(dyn, n["h"], c["nw"], dh=c["dy"])
    # against the same chain in float64 from the kernels' own y and expert outputs
    lf, idn = host(logits), r["topk_ids"].cpu().numpy()
    dwr, _, _ = OL.combine_backward(host(c["dy"]), host(eo), r["assign_pos"].cpu().numpy(), host(r["topk_weights"]))
    ref, mag = OL.route_backward(lf, idn, k, "softmax", True, 1.0, dwr, loss["counts"].cpu().numpy(), CA, CZ)
    # (dweights carry at most (512 / 64 + 32) u of their absolute products, far below 1e-4 of a row)
    assert np.abs(host(d) - ref).max() <= 1e-4 * np.abs(ref).max()
    dx, dw, _, _ = OL.rmsnorm_backward(host(dyn), host(n["h"]), host(c["nw"]), 1e-6, host(c["dy"]))
    assert np.abs(host(back["dx"]) - dx).max() <= 1.5 * UB * np.abs(dx).max()
    assert np.abs(host(back["dweight"]) - dw).max() <= 1e-5 * np.abs(dw).max()


def _all_calls(c):
    """Every operator on one layer's data, each as an object, in the order of use."""
    p, T, k = c["p"], c["T"], c["k"]
    xq, xs = M.moe_quant_act(c["x"])
    lin = M.MoeLinear(xq, xs, c["wo"], residual=c["res"])
    norm = M.MoeAddRmsNorm(lin.y, c["nw"], residual=c["x"], quant=c["quant"])
    g = rng(16)
    logits, _ = f32(g.standard_normal((T, p.num_experts)))
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    off = torch.tensor([0, 30, 30, T - 5], dtype=torch.int32, device=DEV)
    dw, _ = f32(g.standard_normal((T, k)))
    loss = M.MoeBalanceLoss(p, logits, ids, off, CA, CZ)
    eo, _ = f32(g.standard_normal((T * k, c["x"].shape[1])))
    pos = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    comb = M.MoeCombineBackward(c["dy"], eo, pos, dw, d_expert_out=True)
    route = M.MoeRouteBackward(p, logits, ids, comb.out["dweights"], loss.counts, off, CA, CZ)
    nb = M.MoeAddRmsNormBackward(c["dy"], norm.h, c["nw"], dh=c["x"])
    calls = [lin, norm, loss, comb, route, nb]
    outs = [lin.y, norm.h, norm.y, norm.yq, norm.ys, loss.losses, loss.counts, loss.mean_probs, comb.out["dweights"],
            comb.out["d_expert_out"], route.dlogits, nb.out["dx"], nb.out["dweight"]]
    return calls, outs, (logits, dw, c)


@pytest.mark.parametrize("T,N", [(100, 512), (300, 1024), (700, 4096), (2000, 4096), (3000, 6144)])
def test_linear_variants_in_a_graph(T, N):
    """First call under capture (nothing is set up before it), then replays against eager calls."""
    xq, xs, w, _, _ = _linear_inputs(T, 384, N, "fp8", 6)
    res, _ = bf16(rng(18, T, N).standard_normal((T, N)))
    f = M.MoeLinear(xq, xs, w, residual=res)
    g = M.MoeLinear(xq, xs, w, residual=res)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            f()
    for _ in range(3):
        res.mul_(-1.5)
        f.y.zero_()
        graph.replay()
        want = g()
        torch.cuda.synchronize()
        assert torch.equal(f.y, want)


def test_graph_replays_match_eager_calls():
    c = _layer("fp8")
    calls, outs, (logits, dw, _) = _all_calls(c)
    other, other_outs, _ = _all_calls(c)
    for f in calls:
        f()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            for f in calls:
                f()
    torch.cuda.synchronize()
    for rep in range(4):
        with torch.no_grad():
            c["x"].mul_(-0.5)       # new inputs in the same buffers
            logits.add_(0.25 * torch.sin(logits * (rep + 1)))
            c["dy"].neg_()
        for f in other:     # eager calls on other inputs and workspaces between the replays
            f()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for f in calls:
            f()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, outs)):
            assert torch.equal(a, b), (rep, i)
    del graph


def test_side_stream_and_explicit_stream():
    c = _layer("fp8")
    calls, outs, _ = _all_calls(c)
    for f in calls:
        f()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for how in ("current", "explicit"):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if how == "current":
            with torch.cuda.stream(side):
                for f in calls:
                    f()
        else:
            for f in calls:
                f(side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), how


def test_outputs_stay_inside_their_buffers():
    """Guard bands around every output and workspace."""
    T, H, K, N, E, k, S = 137, 520, 384, 208, 21, 3, 3
    g = rng(17)
    x, _ = bf16(g.standard_normal((T, H)))
    w, _ = f32(g.standard_normal(H))
    nb = M.MoeAddRmsNormBackward(x, x, w, dh=x)
    ws = nb.args.workspace_bytes // 256 * 256
    need = B.lib().moe_add_rmsnorm_backward_workspace_size(T, H)
    ar = Arena([T * H * 2, H * 4, need])
    nb.args.dx, nb.args.dweight, nb.args.workspace, nb.args.workspace_bytes = ar.ptr(0), ar.ptr(1), ar.ptr(2), need
    ref = M.moe_add_rmsnorm_backward(x, x, w, dh=x)
    nb()
    ar.assert_guards("norm backward")
    assert torch.equal(ar.view(0, torch.bfloat16, (T, H)), ref["dx"]) and torch.equal(ar.view(1, torch.float32, (H,)), ref["dweight"])
    for hh, quant, gs in ((384, M.MOE_QUANT_FP8_BLOCK128, 128), (544, M.MOE_QUANT_MXFP8, 32)):
        xx, _ = bf16(g.standard_normal((T, hh)))
        ww, _ = f32(g.standard_normal(hh))
        nf = M.MoeAddRmsNorm(xx, ww, residual=xx, quant=quant)
        ref = {n: v.clone() for n, v in nf().items()}
        ar = Arena([T * hh * 2, T * hh * 2, T * hh, T * hh // gs])
        nf.args.h, nf.args.y, nf.args.yq, nf.args.ys = (ar.ptr(i) for i in range(4))
        nf()
        ar.assert_guards("norm")
        assert torch.equal(ar.view(3, torch.uint8, (T, hh // gs)), ref["ys"])
    for TT, KK, NN, scheme in ((T, K, N, "fp8"), (1, K, N, "mxfp8"), (30, K, N, "fp8"), (700, 256, 528, "mxfp8"),
                               (2100, 256, 2064, "fp8")):
        xq, xs, lw, _, _ = _linear_inputs(TT, KK, NN, scheme, 5)
        for dt, size in ((torch.bfloat16, 2), (torch.float32, 4)):
            f = M.MoeLinear(xq, xs, lw, "silu", out_dtype=dt)
            ref = f().clone()
            wsn = B.lib().moe_linear_workspace_size(TT, KK, NN, lw.quant)
            ar = Arena([TT * NN * size, max(wsn, 16)])
            f.args.y = ar.ptr(0)
            if wsn:
                f.args.workspace, f.args.workspace_bytes = ar.ptr(1), wsn
            f()
            ar.assert_guards(f"linear {TT} {KK} {NN}")
            assert torch.equal(ar.view(0, dt, (TT, NN)), ref)
    l, _, ids, _, dw, _ = _router_inputs(T, E, k, 6)
    off = _off([0, 50, 50, 130])
    p = _params(E, k, "softmax", True)
    f = M.MoeBalanceLoss(p, l, ids, off, CA, CZ)
    ref = {n: v.clone() for n, v in f().items()}
    need = B.lib().moe_balance_loss_workspace_size(T, E, S)
    ar = Arena([12, S * E * 4, S * E * 4, need])
    f.args.losses, f.args.counts, f.args.mean_probs, f.args.workspace = (ar.ptr(i) for i in range(4))
    f.args.workspace_bytes = need
    f()
    ar.assert_guards("balance")
    assert torch.equal(ar.view(0, torch.float32, (3,)), ref["losses"]) and torch.equal(ar.view(1, torch.int32, (S, E)), ref["counts"])
    f = M.MoeRouteBackward(p, l, ids, dw, ref["counts"], off, CA, CZ)
    ref = f().clone()
    ar = Arena([T * E * 4])
    f.args.dlogits = ar.ptr(0)
    f()
    ar.assert_guards("route backward")
    assert torch.equal(ar.view(0, torch.float32, (T, E)), ref)
    eo, _ = bf16(g.standard_normal((T * k, 264)))
    dy, _ = bf16(g.standard_normal((T, 264)))
    pos = torch.randperm(T * k, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
    f = M.MoeCombineBackward(dy, eo, pos, dw, d_expert_out=True)
    ref = {n: v.clone() for n, v in f().items()}
    ar = Arena([T * k * 4, T * k * 264 * 2])
    f.args.dtopk_weights, f.args.dexpert_out = ar.ptr(0), ar.ptr(1)
    f()
    ar.assert_guards("combine backward")
    assert torch.equal(ar.view(1, torch.bfloat16, (T * k, 264)), ref["d_expert_out"])


def test_binding_refuses():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, device=DEV)
    with pytest.raises(TypeError):
        M.moe_add_rmsnorm(x.float(), w)
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(x, w[:128])
    with pytest.raises(TypeError):
        M.moe_add_rmsnorm(x, w.cpu())
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(x.t().contiguous().t(), w)
    with pytest.raises(M.MoeError):
        M.moe_add_rmsnorm(x[:1].expand(4, 256), w)             # rows on top of each other: ld 0
    with pytest.raises(M.MoeError):
        M.moe_add_rmsnorm(x[:, :100].contiguous(), w[:100].contiguous())   # H % 8
    with pytest.raises(M.MoeError):
        M.moe_add_rmsnorm(x, w, want_y=False)                  # nothing to compute
    xq, xs = M.moe_quant_act(x)
    lw = M.LinearWeights.from_float(torch.zeros(256, 128, device=DEV))
    for bad in (dict(K=128), dict(N=256), dict(w_scale=lw.w_scale[:1]), dict(bias=torch.zeros(64, device=DEV))):
        with pytest.raises(ValueError):
            M.moe_linear(xq if "K" not in bad else xq[:, :128].contiguous(), xs if "K" not in bad else xs[:, :1].contiguous(),
                         dataclasses.replace(lw, **bad))
    with pytest.raises(TypeError):
        M.moe_linear(xq, xs, dataclasses.replace(lw, w=lw.w.cpu()))
    with pytest.raises(TypeError):
        M.moe_linear(xq, xs, lw, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        M.moe_linear(xq, xs, lw, "swish")
    with pytest.raises(ValueError):
        M.moe_linear(xq, xs[:, :1].contiguous(), lw)
    with pytest.raises(ValueError):
        M.moe_linear(xq, xs, lw, residual=torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        M.moe_linear(xq, xs, lw, residual=torch.zeros(4, 128, device=DEV))
    with pytest.raises(ValueError):
        M.LinearWeights.from_logical(torch.zeros(256, 128, dtype=torch.uint8, device=DEV),
                                     torch.zeros(2, 1, dtype=torch.uint8, device=DEV), M.MOE_QUANT_W4A8)
    p = M.route_params(8, 2)
    l = torch.zeros(4, 8, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        M.moe_balance_loss(p, l, ids, torch.zeros(1, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        M.moe_balance_loss(p, l, ids.long())
    with pytest.raises(ValueError):
        M.moe_route_backward(p, l, None, torch.zeros(4, 2, device=DEV))
    with pytest.raises(ValueError):
        M.moe_combine_backward(x, torch.zeros(8, 256, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV),
                               torch.zeros(4, 2, device=DEV))
