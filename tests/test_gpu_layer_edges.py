"""Edges of the operators around the expert step on the GPU: infinite weights, the far tail of GELU,
a handle whose assignments change from call to call, more rows than one launch holds, very many
sequences, and the kernel variants that only large calls reach.

Tolerances as in test_gpu_layer.py: u = 2^-24 is half a float32 step, 2^-8 half a bf16 step."""
import numpy as np
import pytest
import torch

import test_gpu_layer as GL
from oracle import layer as OL
from oracle.w8a16 import bf16_rne
from test_gpu_layer import DEV, M, TINY, U, UB, bf16, f32, host, rng, within

pytestmark = pytest.mark.gpu


# ---- residual + RMS norm ------------------------------------------------------------------
@pytest.mark.parametrize("H,quant", [(256, "fp8"), (544, "mxfp8"), (4104, None), (7168, "fp8")])
def test_add_rmsnorm_infinite_weights(H, quant):
    """A weight of either infinity gives the infinity that h's sign asks for, and NaN where h is 0."""
    h, hf = bf16(rng(31, H).standard_normal((5, H)))
    h[:, 11] = 0
    hf[:, 11] = 0
    w, wf = f32(1 + 0.1 * rng(32, H).standard_normal(H))
    for c, v in ((3, np.inf), (8, -np.inf), (11, np.inf), (H - 1, -np.inf), (40, np.finfo(np.float32).max)):
        w[c], wf[c] = float(v), v
    h[:, 40], hf[:, 40] = 3.0, 3.0         # a finite product past the largest bf16 value
    out = M.moe_add_rmsnorm(h, w, 1e-6, quant=None if quant is None else M.QUANT_SCHEMES[quant])
    _, y = OL.add_rmsnorm(hf, None, wf, 1e-6)
    assert np.isnan(y[:, 11]).all() and np.isinf(y[:, [3, 8, H - 1]]).all()
    with np.errstate(over="ignore"):
        want = bf16_rne(y)
    got = host(out["y"])
    assert np.array_equal(np.isnan(got), np.isnan(y))
    ends = [3, 8, 40, H - 1]
    assert np.array_equal(got[:, ends], np.sign(want[:, ends]) * np.inf)
    if quant:
        q, s = M.moe_quant_act(out["y"]) if quant == "fp8" else M.moe_quant_act_mx(out["y"])
        assert torch.equal(out["yq"], q) and torch.equal(out["ys"], s)


# Matrices of 32 MiB and more go past the caches, by kernels of their own.
@pytest.mark.parametrize("T,H,quant,residual", [(4097, 4104, None, True), (2400, 7168, "mxfp8", True), (2341, 7168, "fp8", False),
                                                (33000, 512, "fp8", True), (8200, 2048, "mxfp8", True), (1025, 16384, None, True),
                                                (513, 32768, "fp8", True)])
def test_add_rmsnorm_streamed(T, H, quant, residual):
    x, xf, r, rf, w, wf = GL._norm_inputs(T, H, 5)
    out = M.moe_add_rmsnorm(x, w, 1e-6, residual=r if residual else None, quant=None if quant is None else M.QUANT_SCHEMES[quant])
    h, y = OL.add_rmsnorm(xf, rf if residual else None, wf, 1e-6)
    if residual:
        assert np.array_equal(host(out["h"]), h)
    # (bounds as in test_add_rmsnorm)
    near = bf16_rne(y * (1 + 2.0 ** -30)) != bf16_rne(y * (1 - 2.0 ** -30))
    assert np.array_equal(host(out["y"])[~near], bf16_rne(y)[~near]) and near.mean() < 1e-4
    if quant:
        q, s = M.moe_quant_act(out["y"]) if quant == "fp8" else M.moe_quant_act_mx(out["y"])
        assert torch.equal(out["yq"], q) and torch.equal(out["ys"], s)
    # the last rows alone, by the kernels of small matrices: the same bits
    few = M.moe_add_rmsnorm(x[-3:], w, 1e-6, residual=r[-3:] if residual else None)
    assert torch.equal(few["y"], out["y"][-3:])


# Several rows per workgroup in every kernel, both numbers of workgroups, and streamed matrices.
@pytest.mark.parametrize("T,H", [(700, 1544), (700, 2816), (600, 7168), (4500, 1544), (33000, 40), (33000, 512), (2600, 1000),
                                 (4200, 4096), (2400, 7168), (8300, 2048), (1100, 16384), (600, 32768), (17000, 1024)])
def test_add_rmsnorm_backward_many_rows(T, H):
    GL.test_add_rmsnorm_backward(T, H, T % 3 != 0)


# ---- linear -------------------------------------------------------------------------------
def _tail(name, v):
    """The activation in 64 bits without the cancellation of 1 + erf(v / sqrt 2) and 1 + tanh u."""
    from scipy.special import ndtr
    if name == "gelu":
        return v * ndtr(v)
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    u = np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)
    return v / (1.0 + np.exp(-2.0 * u))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T,N", [(1, 8192), (80, 8192), (600, 4096), (2100, 8192)])
def test_linear_activation_tails(act, T, N):
    """Relative to the activation's own value, also where that is small.  With rows of zeros the sum is
    0 and the activation's argument is the bias itself."""
    w = M.LinearWeights.from_float(torch.zeros(128, N, device=DEV))
    v, vf = f32(np.concatenate([np.linspace(-12.8, -0.01, N // 2), np.linspace(1e-3, 9.0, N // 2)]))
    w.bias = v
    xq, xs = M.moe_quant_act(torch.zeros(T, 128, dtype=torch.bfloat16, device=DEV))
    want = _tail(act, vf)[None]
    # The exponent x is off by 3 u |x| (a product or two and a constant), which is the relative error of
    # exp x: |x| is v^2 / 2, |2 u(v)| (whose argument adds another 4 u) and |v|.  Beside it: reciprocal and
    # exponential instructions (one unit in the last place, 2 u each), the polynomial of GELU (fit 3 u,
    # eight terms of one size 8 u, its argument's 6 u) and the last products.
    x = {"gelu": 0.5 * vf ** 2, "silu": np.abs(vf),
         "gelu_tanh": 2 * np.abs(np.sqrt(2 / np.pi) * (vf + 0.044715 * vf ** 3)) * 7 / 3}[act][None]
    rel = (3 * x + 32) * U
    for dt in (torch.float32, torch.bfloat16):
        got = host(M.moe_linear(xq, xs, w, act, out_dtype=dt))
        tol = rel * np.abs(want) + 2.0 ** -122 + (UB * np.abs(want) * (1 + rel) if dt == torch.bfloat16 else 0)
        within(got, np.broadcast_to(want, got.shape), np.broadcast_to(tol, got.shape), f"{act} {dt}")


# ---- combine --------------------------------------------------------------------------------
def _combine_inputs(T, k, H, dtype, key):
    g = rng(33, T, k, H, key)
    mk = bf16 if dtype == "bf16" else f32
    return mk(g.standard_normal((T * k, H)))[0], bf16(g.standard_normal((T, H)))[0], f32(g.random((T, k)))[0], g


def _rows_of(pos, T, k, H, w, dy, dtype):
    """d_expert_out: the named rows' gradients (one float32 product, then rounded to dtype), zeros beside them."""
    want = torch.zeros(T * k, H, dtype=dtype, device=DEV)
    f = np.nonzero((pos >= 0) & (pos < T * k))[0]
    rows, f = torch.from_numpy(pos[f].astype(np.int64)).to(DEV), torch.from_numpy(f).to(DEV)
    want[rows] = (w.reshape(-1)[f, None] * dy.float()[f // k]).to(dtype)
    return want


COMBINE_EDGES = [(1, 1, 8, "bf16"), (5, 8, 1024, "bf16"), (4, 9, 1032, "f32"), (300, 8, 264, "bf16"), (300, 3, 4096, "f32"),
                 (4099, 2, 1032, "bf16"), (4099, 1, 264, "f32"), (70000, 1, 8, "bf16"), (2100, 10, 72, "f32"),
                 (40001, 2, 128, "bf16")]


@pytest.mark.parametrize("T,k,H,dtype", COMBINE_EDGES)
def test_combine_handle_with_changing_assignments(T, k, H, dtype):
    """Rows that a later call no longer names hold that call's gradient, 0, not an earlier one's."""
    eo, dy, w, g = _combine_inputs(T, k, H, dtype, 1)
    A = T * k
    at = T % 4                      # (entries at any 4-byte address)
    pos = torch.zeros(A + 4, dtype=torch.int32, device=DEV)[at:at + A]
    pos.copy_(torch.from_numpy(g.permutation(A).astype(np.int32)))
    call = M.MoeCombineBackward(dy, eo, pos, w, d_expert_out=True)
    for share in (0.0, 0.3, 0.9, 1.0, 0.05):
        p = g.permutation(A).astype(np.int32)
        p[g.random(A) < share] = -1
        if share == 0.3:
            p[p == -1] = A + 5      # (past the end is dropped as well)
        pos.copy_(torch.from_numpy(p))
        out = call()
        want = _rows_of(p, T, k, H, w, dy, eo.dtype)
        assert torch.equal(out["d_expert_out"], want), share
        assert torch.equal(M.moe_combine_backward(dy, eo, pos, w, d_expert_out=True)["d_expert_out"], want)
    # whatever the buffer held
    call.out["d_expert_out"].fill_(float("nan"))
    assert torch.equal(call()["d_expert_out"], want)
    # a caller's own tensor keeps its other rows
    mine = torch.full_like(eo, 3.0)
    M.moe_combine_backward(dy, eo, pos, w, d_expert_out=mine)
    named = torch.zeros(A, dtype=torch.bool, device=DEV)
    named[pos[(pos >= 0) & (pos < A)].long()] = True
    assert (mine[~named] == 3.0).all() and torch.equal(mine[named], want[named])


def test_combine_handle_with_changing_assignments_in_a_graph():
    T, k, H = 500, 4, 520
    eo, dy, w, g = _combine_inputs(T, k, H, "bf16", 2)
    pos = torch.from_numpy(g.permutation(T * k).astype(np.int32)).to(DEV)
    call = M.MoeCombineBackward(dy, eo, pos, w, d_expert_out=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    for share in (0.5, 0.0, 0.9, 0.2):
        p = g.permutation(T * k).astype(np.int32)
        p[g.random(T * k) < share] = -1
        pos.copy_(torch.from_numpy(p))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out["d_expert_out"], _rows_of(p, T, k, H, w, dy, eo.dtype)), share
        M.moe_combine_backward(dy, eo, pos, w)
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,k,H,dtype", [(4099, 2, 1032, "bf16"), (4100, 1, 264, "f32"), (1025, 2, 1100 * 8, "bf16"), (200, 3, 2064, "f32")])
def test_combine_backward_variants(T, k, H, dtype):
    GL.test_combine_backward(T, k, H, dtype)


# ---- more rows than one launch of a thread group per row may hold ------------------------------
def test_more_rows_than_one_launch():
    """HIP refuses a launch of 2^32 threads: a wave per row of 8 columns comes to that at 2^26 rows."""
    H, T = 8, (1 << 26) + 3
    pick = torch.tensor([0, 1, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, (1 << 26) - 1, 1 << 26, T - 1], device=DEV)
    x = torch.randn(T, H, device=DEV, dtype=torch.bfloat16)
    w, _ = f32(1 + 0.1 * rng(34).standard_normal(H))
    print("norm", flush=True)
    out = M.moe_add_rmsnorm(x, w, 1e-6, residual=x)
    few = M.moe_add_rmsnorm(x[pick].contiguous(), w, 1e-6, residual=x[pick].contiguous())
    assert torch.equal(out["y"][pick], few["y"]) and torch.equal(out["h"][pick], few["h"])
    assert torch.equal(out["h"], x + x) and torch.isfinite(out["y"]).all()
    del out
    print("norm backward", flush=True)
    d = M.moe_add_rmsnorm_backward(x, x, w, 1e-6, want_dweight=False)["dx"]
    assert torch.equal(d[pick], M.moe_add_rmsnorm_backward(x[pick].contiguous(), x[pick].contiguous(), w, 1e-6, want_dweight=False)["dx"])
    del d
    print("combine", flush=True)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    cw = torch.rand(T, 1, device=DEV)
    c = M.moe_combine_backward(x, x, pos, cw, d_expert_out=True)
    assert torch.equal(c["d_expert_out"], (cw * x.float()).to(torch.bfloat16).flip(0))
    dots = (x[pick].double() * x.flip(0)[pick].double()).sum(1)
    mag = (x[pick].double() * x.flip(0)[pick].double()).abs().sum(1)
    within(host(c["dweights"][pick, 0]), host(dots), 40 * U * host(mag))
    pos[5] = -1
    c = M.moe_combine_backward(x, x, pos, cw, d_expert_out=True)
    assert (c["d_expert_out"][T - 6] == 0).all() and c["dweights"][5, 0] == 0


def test_more_router_rows_than_one_launch():
    """16 lanes per row: 2^32 threads at 2^28 rows."""
    T, E, k = (1 << 28) + 5, 2, 1
    l = torch.randn(T, E, device=DEV)
    pick = torch.tensor([0, 15, 16, (1 << 27) - 1, 1 << 27, (1 << 28) - 1, 1 << 28, T - 1], device=DEV)
    p = GL._params(E, k, "softmax", True)
    d = M.moe_route_backward(p, l, None, None, None, None, 0.0, 1.0)
    sub = l[pick].double()
    lse = torch.logsumexp(sub, 1, keepdim=True)
    want = 2.0 / T * lse * torch.softmax(sub, 1)
    assert ((d[pick].double() - want).abs() <= 1e-5 * want.abs() + 1e-13).all()
    del l
    assert torch.isfinite(d).all() and (d != 0).any(1).float().mean() > 0.999


# ---- very many sequences -----------------------------------------------------------------------
def _us(f, n=3):
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("E", [8, 300])
def test_route_backward_with_very_many_sequences(E):
    """A sequence per row, up to the limit: right, and not a walk over all boundaries for every 16 rows."""
    T, k = 1 << (20 if E == 8 else 16), 2
    l, lf, ids, idn, dw, dwf = GL._router_inputs(T, E, k, 21)
    off = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    p = GL._params(E, k, "softmax", True, 1.3)
    counts = torch.zeros(T, E, dtype=torch.int32, device=DEV).scatter_(1, ids.long(), 1)
    d = M.moe_route_backward(p, l, ids, dw, counts, off, 0.5, 0.1)
    s = torch.softmax(l.double(), 1)
    u = 0.5 / T * E / k * counts.double()
    want = s * (u - (s * u).sum(1, keepdim=True)) + 0.2 / T * torch.logsumexp(l.double(), 1, keepdim=True) * s
    mag = s * (u + (s * u).sum(1, keepdim=True)) + 0.2 / T * torch.logsumexp(l.double(), 1, keepdim=True).abs() * s
    q = torch.softmax(torch.gather(l.double(), 1, ids.long()), 1)
    want = want.scatter_add(1, ids.long(), 1.3 * q * (dw.double() - (q * dw.double()).sum(1, keepdim=True)))
    mag = mag.scatter_add(1, ids.long(), 1.3 * q * (dw.double().abs() + (q * dw.double().abs()).sum(1, keepdim=True)))
    R = float(l.max() - l.min())
    within(host(d), host(want), (4 * (R + 40) + 128) * U * host(mag) + 1e-12)
    only = M.MoeRouteBackward(p, l, ids, dw, None, off, 0.0, 0.0)
    full = M.MoeRouteBackward(p, l, ids, dw, counts, off, 0.5, 0.1)
    one = M.MoeRouteBackward(p, l, ids, dw, None, None, 0.0, 0.0)
    only(), full(), one()
    t = [_us(only), _us(full), _us(one)]
    print("weights alone, everything, one sequence: %.0f %.0f %.0f us" % tuple(t), flush=True)
    assert t[0] < 10 * t[2] + 1000 and t[1] < 12000      # (one workgroup per 16 rows: 33900 us each)


@pytest.mark.parametrize("S", [1024, 1025, 3000])
def test_route_backward_sequences_around_the_table(S):
    """Boundaries held in LDS and searched in memory; uneven lengths, empty sequences, rows outside."""
    T = 9000
    g = rng(35, S)
    off = np.sort(g.integers(3, T - 40, S + 1))
    off[10:30] = off[10]
    GL.test_balance_loss_and_route_backward(T, 24, 3, "softmax", True, 1.5, [int(o) for o in off])


@pytest.mark.parametrize("T,E,k,scoring", [(40000, 60, 4, "softmax"), (40000, 67, 3, "sigmoid"), (33000, 128, 8, "softmax"),
                                           (33000, 130, 8, "sigmoid"), (33000, 256, 20, "softmax"), (8300, 260, 5, "softmax"),
                                           (8300, 513, 70, "sigmoid"), (8300, 1001, 12, "softmax"), (8300, 1024, 8, "sigmoid")])
def test_route_backward_rows_in_turn(T, E, k, scoring):
    """Workgroups that take several rows (more sequences than LDS holds, and counts): the same bits as one row
    each, which the same boundaries take without the empty sequences behind them."""
    l, _, ids, _, dw, _ = GL._router_inputs(T, E, k, 22)
    off = np.sort(rng(36, T, E).integers(0, T + 1, 1025)).astype(np.int32)
    more = np.concatenate([off, np.full(200, off[-1], dtype=np.int32)])
    p = GL._params(E, k, scoring, True, 0.8)
    few = M.moe_balance_loss(p, l, ids, torch.from_numpy(off).to(DEV), 0.3, 0.02)
    many = M.moe_balance_loss(p, l, ids, torch.from_numpy(more).to(DEV), 0.3, 0.02)
    assert torch.equal(many["counts"][:1024], few["counts"]) and (many["counts"][1024:] == 0).all()
    a = M.moe_route_backward(p, l, ids, dw, few["counts"], torch.from_numpy(off).to(DEV), 0.3, 0.02)
    b = M.moe_route_backward(p, l, ids, dw, many["counts"], torch.from_numpy(more).to(DEV), 0.3, 0.02)
    assert torch.equal(a, b) and (a != 0).any()
