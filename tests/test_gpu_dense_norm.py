"""Residual + layer norm and its backward pass on the GPU against the float64 oracle (oracle/dense.py);
tolerances as in test_gpu_layer.py."""
import numpy as np
import pytest
import torch

import harness as HN
from oracle import dense as OD
from oracle.w8a16 import bf16_rne
from test_gpu_guards import Arena
from test_gpu_layer import TINY, U, UB, _check_codes, bf16, f32, host, rng, strided, within

pytestmark = pytest.mark.gpu

M = pytest.importorskip("mixture_experts_fp8_amd")
B = M.binding

CASES = [  # T, H, quant, residual, bias, stride padding
    (1, 128, "fp8", True, True, 0), (1, 8, None, True, True, 0), (3, 136, None, False, True, 8),
    (5, 512, "mxfp8", True, False, 0), (7, 520, None, True, True, 16), (32, 2816, "fp8", True, True, 0),
    (9, 768, "w4a8", False, True, 0), (33, 4096, "fp8", False, False, 8), (4, 4104, None, True, True, 0),
    (6, 7168, "mxfp8", True, True, 8), (3, 8224, "mxfp8", False, True, 0), (2, 16512, "fp8", True, True, 0),
    (1, 32768, "mxfp8", True, True, 0), (257, 256, "fp8", True, True, 0),
    (2500, 7168, "mxfp8", True, True, 0),     # past the caches
]


def _inputs(T, H, key, shift=0.5):
    g = rng(17, T, H, key)
    x, xf = bf16(g.standard_normal((T, H)) * np.where(g.random(H) < 0.02, 20.0, 1.0) + shift)
    r, rf = bf16(g.standard_normal((T, H)))
    w, wf = f32(1 + 0.1 * g.standard_normal(H))
    b, bf = f32(0.1 * g.standard_normal(H))
    return x, xf, r, rf, w, wf, b, bf


@pytest.mark.parametrize("T,H,quant,residual,bias,pad", CASES)
def test_add_layernorm(T, H, quant, residual, bias, pad):
    x, xf, r, rf, w, wf, b, bf = _inputs(T, H, 1)
    b, bf = (b, bf) if bias else (None, None)
    xs, rs = (strided(x, pad), strided(r, pad)) if pad else (x, r)
    q = None if quant is None else M.QUANT_SCHEMES[quant]
    out = M.moe_add_layernorm(xs, w, b, 1e-5, residual=rs if residual else None, quant=q)
    h, y = OD.add_layernorm(xf, rf if residual else None, wf, bf, 1e-5)
    if residual:
        assert np.array_equal(host(out["h"]), h)
    else:
        assert out["h"] is None
    # y is formed in double: H additions of d and d^2 whose variance loses at most a factor H, 2^15, of
    # 2^-53 (H + 8), then the products and the bias, whose terms may cancel: below 2^-28 of |y| + |bias|
    # (inputs here keep the factor far below H).  Rounded once: the definition's bf16 value, but for values that
    # near to a tie
    off = 2.0 ** -28 * (np.abs(y) + (0 if bf is None else np.abs(bf)))
    near = bf16_rne(y + off) != bf16_rne(y - off)
    assert np.array_equal(host(out["y"])[~near], bf16_rne(y)[~near]) and near.mean() < 1e-4
    if quant:
        _check_codes(out, out["y"], quant)
    again = M.moe_add_layernorm(xs, w, b, 1e-5, residual=rs if residual else None, want_y=False, quant=q,
                                h=torch.empty_like(x) if quant is None else None)
    assert again["y"] is None and (quant is None or torch.equal(again["yq"], out["yq"]))
    if residual and not pad:        # h over the residual, then over x
        for over in ("residual", "x"):
            a, c = x.clone(), r.clone()
            got = M.moe_add_layernorm(a, w, b, 1e-5, residual=c, h=c if over == "residual" else a)
            assert torch.equal(got["h"], out["h"]) and torch.equal(got["y"], out["y"])
            assert torch.equal(a if over == "residual" else c, x if over == "residual" else r)
    if not residual and not pad:
        a = x.clone()
        assert torch.equal(M.MoeAddLayerNorm(a, w, b, 1e-5, y=a)()["y"], out["y"])


def test_add_layernorm_special_rows():
    """Rows of one value (also a large one, and where H is no power of two), rows far from 0 with the smallest
    possible spread, the ends of the range, infinities and NaN, each in its own row."""
    H = 264
    g = rng(18)
    v = g.standard_normal((9, H))
    v[0] = 0
    v[1] = 1e30
    v[2] = 100.0 + (np.arange(H) % 2) * 0.5       # a bf16 step apart
    v[3] = 100.0
    v[3, 0] = 100.5                               # all but the first value equal
    v[4] *= 1e-38
    v[5] *= 1e30
    v[6, 5] = np.inf
    v[7, 7] = np.nan
    x, xf = bf16(v)
    w, wf = f32(1 + 0.1 * g.standard_normal(H))
    b, bf = f32(g.standard_normal(H))
    y = host(M.moe_add_layernorm(x, w, b, 1e-5)["y"])
    assert np.array_equal(y[0], bf16_rne(bf)) and np.array_equal(y[1], bf16_rne(bf))
    assert np.isnan(y[6]).all() and np.isnan(y[7]).all()
    fine = [2, 3, 4, 5, 8]
    _, ref = OD.add_layernorm(xf[fine], None, wf, bf, 1e-5)
    within(y[fine], ref, np.abs(ref) * UB + 2.0 ** -28 * (np.abs(ref) + np.abs(bf)) + TINY)
    # eps = 0: 0 / 0 in a row of equal values, as in the formula
    assert np.isnan(host(M.moe_add_layernorm(x, w, b, 0.0)["y"][:2])).all()
    assert np.isfinite(host(M.moe_add_layernorm(x, w, b, 0.0)["y"][2:4])).all()


BWD = [(1, 128), (1, 8), (2, 64), (5, 512), (4999, 184), (9000, 16), (3, 136), (5, 520), (40, 2816), (33, 4096), (4, 4104),
       (6, 7168), (2, 8224), (3, 16512), (1, 32768), (513, 256), (1100, 64), (1537, 1024), (7, 600), (2100, 968),
       (300, 16400), (290, 10000), (4200, 4096)]


@pytest.mark.parametrize("T,H", BWD)
@pytest.mark.parametrize("with_dh", [True, False])
def test_add_layernorm_backward(T, H, with_dh):
    x, xf, r, rf, w, wf, _, _ = _inputs(T, H, 2)
    dy, dyf = bf16(0.1 * rng(19, T, H).standard_normal((T, H)))
    out = M.moe_add_layernorm_backward(dy, x, w, 1e-5, dh=r if with_dh else None)
    dx, dw, db, mag, dwmag, dbmag = OD.layernorm_backward(dyf, xf, wf, 1e-5, rf if with_dh else None)
    # dx: means and xhat in double, of h - h[0] and g in float32 (1 u each).  In float32: mean(g), xhat and
    # mean(g xhat) rounded (1 u each), xhat mean(g xhat) and two subtractions, the product with r and r itself, the addition of
    # dh: no term of `mag` passes more than 10 roundings.  Then the rounding to bf16.
    within(host(out["dx"]), dx, UB * np.abs(dx) + 10 * U * (1 + UB) * mag + TINY, "dx")
    # the sums over rows, of xhat off by 3 u (h - h[0], which is at most 2 (|xhat| + 1) standard deviations for these h[0],
    # and its rounding): a workgroup's rows in turn, then the partial rows (a 32nd of them in a chain, 32 chains)
    parts = B.lib().moe_add_layernorm_backward_workspace_size(T, H) // (8 * H)
    chain = -(-T // parts) + 4 + -(-parts // 32) + 32
    within(host(out["dweight"]), dw, (chain + 8) * U * dwmag + 8 * U * dbmag + 1e-38, "dweight")
    within(host(out["dbias"]), db, (chain + 4) * U * dbmag + 1e-38, "dbias")
    again = M.moe_add_layernorm_backward(dy, x, w, 1e-5, dh=r if with_dh else None)
    assert all(torch.equal(again[n], out[n]) for n in out)
    # each vector alone or none, in place over dy and over dh
    for want in ((True, False), (False, True), (False, False)):
        a = dy.clone()
        got = M.MoeAddLayerNormBackward(a, x, w, 1e-5, dh=r if with_dh else None, want_dweight=want[0],
                                        want_dbias=want[1], dx=a)()
        assert torch.equal(a, out["dx"])
        for on, n in zip(want, ("dweight", "dbias")):
            assert got[n] is None if not on else torch.equal(got[n], out[n])
    if with_dh:
        c = r.clone()
        M.MoeAddLayerNormBackward(dy, x, w, 1e-5, dh=c, dx=c)()
        assert torch.equal(c, out["dx"])


@pytest.mark.parametrize("H", [64, 1000, 4096, 20000])
def test_add_layernorm_backward_special_rows(H):
    """Rows whose squares leave float32 on either side, far from 0 against their spread, of one value,
    infinite, NaN."""
    g = rng(20, H)
    h = g.standard_normal((8, H)) * np.array([1e-30, 1e-15, 1, 1e20, 1e30, 1, 1, 1])[:, None]
    h[5] = 1000 + 4 * (np.arange(H) % 2)
    h[6] = -3.0
    dy, dyf = bf16(g.standard_normal((8, H)))
    h, hf = bf16(h)
    w, wf = f32(1 + 0.1 * g.standard_normal(H))
    out = M.moe_add_layernorm_backward(dy, h, w, 1e-5)
    dx, _, _, mag, _, _ = OD.layernorm_backward(dyf, hf, wf, 1e-5)
    within(host(out["dx"]), dx, UB * np.abs(dx) + 10 * U * (1 + UB) * mag + TINY, "dx")
    for row in range(8):
        one = M.moe_add_layernorm_backward(dy[row:row + 1], h[row:row + 1], w, 1e-5)
        assert torch.equal(one["dx"], out["dx"][row:row + 1])
        _, dw, db, _, dwmag, _ = OD.layernorm_backward(dyf[row:row + 1], hf[row:row + 1], wf, 1e-5)
        within(host(one["dweight"]), dw, 8 * U * (dwmag + np.abs(dyf[row])) + 1e-38, "dweight")
        assert np.array_equal(host(one["dbias"]), db)
    bad = h.clone()
    bad[0, 3], bad[1, 5] = float("inf"), float("nan")
    got = M.moe_add_layernorm_backward(dy, bad, w, 1e-5, dh=dy)["dx"]
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    assert torch.equal(got[2:], M.moe_add_layernorm_backward(dy[2:], h[2:], w, 1e-5, dh=dy[2:])["dx"])


def test_add_layernorm_backward_against_differences():
    g = rng(21)
    h, hf = bf16(g.standard_normal((3, 16)))
    dy, dyf = bf16(g.standard_normal((3, 16)))
    w, wf = f32(g.standard_normal(16))
    out = M.moe_add_layernorm_backward(dy, h, w, 1e-3)
    step = 1e-5
    num = np.zeros_like(hf)
    for i in range(3):
        for j in range(16):
            hi, lo = hf.copy(), hf.copy()
            hi[i, j] += step
            lo[i, j] -= step
            num[i, j] = ((OD.add_layernorm(hi, None, wf, None, 1e-3)[1] - OD.add_layernorm(lo, None, wf, None, 1e-3)[1])
                         * dyf).sum() / (2 * step)
    # the central difference is off by step^2 / 6 of the third derivative: < 1e-7 at these values
    within(host(out["dx"]), num, UB * np.abs(num) + 1e-6)


def test_add_layernorm_stays_inside_its_buffers():
    T, H = 37, 2816
    x, _, r, _, w, _, b, _ = _inputs(T, H, 3)
    want = M.moe_add_layernorm(x, w, b, 1e-5, residual=r, quant=0)
    a = Arena([2 * T * H, 2 * T * H, T * H, T * H // 128])
    call = M.MoeAddLayerNorm(x, w, b, 1e-5, residual=r, quant=0)
    call.args.h, call.args.y, call.args.yq, call.args.ys = (a.ptr(i) for i in range(4))
    call()
    a.assert_guards("layer norm")
    for i, (n, t) in enumerate((("h", torch.bfloat16), ("y", torch.bfloat16), ("yq", torch.uint8), ("ys", torch.uint8))):
        assert torch.equal(a.view(i, t, want[n].shape), want[n])
    dy = r
    full = M.moe_add_layernorm_backward(dy, x, w, 1e-5)
    n = B.lib().moe_add_layernorm_backward_workspace_size(T, H)
    a = Arena([2 * T * H, 4 * H, 4 * H, n])
    call = M.MoeAddLayerNormBackward(dy, x, w, 1e-5)
    call.args.dx, call.args.dweight, call.args.dbias, call.args.workspace = (a.ptr(i) for i in range(4))
    call.args.workspace_bytes = n
    call()
    a.assert_guards("layer norm backward")
    assert torch.equal(a.view(0, torch.bfloat16, (T, H)), full["dx"])
    assert torch.equal(a.view(1, torch.float32, (H,)), full["dweight"])
    assert torch.equal(a.view(2, torch.float32, (H,)), full["dbias"])
    # a single part with buffers at any float: dweight aligned for vectors, dbias not, and the other way round
    for off in ((0, 1), (1, 0), (1, 1)):
        one = M.moe_add_layernorm_backward(dy[:1], x[:1], w, 1e-5)
        f = torch.full((2 * H + 64,), 7.0, device="cuda")
        views = f[off[0]:off[0] + H], f[H + 32 + off[1]:2 * H + 32 + off[1]]
        call = M.MoeAddLayerNormBackward(dy[:1], x[:1], w, 1e-5)
        call.args.dweight, call.args.dbias = views[0].data_ptr(), views[1].data_ptr()
        call()
        assert torch.equal(views[0], one["dweight"]) and torch.equal(views[1], one["dbias"])
        assert (f == 7).sum() == 64
