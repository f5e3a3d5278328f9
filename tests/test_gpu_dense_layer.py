"""The operators of dense layers together, as a model calls them, on the GPU against the float64 oracle; and under
HIP graphs and on other streams.  Tolerances as in test_gpu_layer.py."""
import numpy as np
import pytest
import torch

from oracle import codec, dense as OD, layer as OL, mx, moe as omoe
from oracle.w8a16 import bf16_rne
from test_gpu_layer import TINY, U, UB, bf16, f32, host, rng, within

pytestmark = pytest.mark.gpu

M = pytest.importorskip("mixture_experts_fp8_amd")
B = M.binding
DEV = "cuda"


class _Layer:
    """A dense layer of T rows: norm with codes, gated block, down projection with the residual stream, the
    requests' adapters on it; backward through the block and the norm."""

    def __init__(self, scheme, T=150, H=512, I=384, R=16, n=4, key=1):
        g = rng(71, T, H, I, key)
        self.T, self.H, self.I, self.n = T, H, I, n
        self.scheme, self.quant = scheme, M.QUANT_SCHEMES[scheme]
        self.x, self.xf = bf16(g.standard_normal((T, H)) + 0.3)
        self.res, self.resf = bf16(g.standard_normal((T, H)))
        self.nw, self.nwf = f32(1 + 0.1 * g.standard_normal(H))
        self.nb, self.nbf = f32(0.1 * g.standard_normal(H))
        self.b1, self.b1f = f32(0.1 * g.standard_normal(2 * I))
        w1, w2 = 0.05 * g.standard_normal((H, 2 * I)), 0.05 * g.standard_normal((I, H))
        enc = (lambda w: mx.quant_weight_k32(w, mx.FMT_E4M3)) if scheme == "mxfp8" else codec.quant_blocks_128
        (q1, s1), (q2, s2) = enc(w1), enc(w2)
        up = lambda a: torch.from_numpy(a).to(DEV)
        self.w1 = M.LinearWeights.from_logical(up(q1), up(s1), self.quant, bias=self.b1)
        self.w2 = M.LinearWeights.from_logical(up(q2), up(s2), self.quant)
        self.q = (q1, s1, q2, s2)
        a, self.af = bf16(g.standard_normal((n, R, I)) * I ** -0.5)
        b, self.bf = bf16(g.standard_normal((n, H, R)) * R ** -0.5)
        sc, self.sf = f32(0.5 + g.random(n))
        self.lw = M.LoraWeights(a, b, sc)
        self.off = torch.tensor([0, 1, 1, 40, 41, T - 9], dtype=torch.int32, device=DEV)
        self.ids = torch.tensor([2, 0, 3, -1, 1], dtype=torch.int32, device=DEV)
        self.dh, self.dhf = bf16(0.1 * g.standard_normal((T, I)))
        self.dres, self.dresf = bf16(0.1 * g.standard_normal((T, H)))
        # the calls, each with buffers of its own
        self.norm = M.MoeAddLayerNorm(self.x, self.nw, self.nb, 1e-5, residual=self.res, quant=self.quant)
        self.block = M.MoeGatedLinear(self.norm.yq, self.norm.ys, self.w1, "silu", want_gu=True)
        gs = 32 if scheme == "mxfp8" else 128
        self.hq = torch.empty(T, I, dtype=torch.uint8, device=DEV)
        self.hs = torch.empty(T, I // gs, dtype=torch.uint8, device=DEV)
        self.down = M.MoeLinear(self.hq, self.hs, self.w2, residual=self.norm.h)
        self.lora = M.MoeLora(self.block.h, self.lw, self.ids, self.off, residual=self.down.y, y=self.down.y)
        self.block_bwd = M.MoeGatedLinearBackward(self.dh, self.block.gu, self.w1, self.norm.yq, self.norm.ys, "silu")
        self.norm_bwd = M.MoeAddLayerNormBackward(self.block_bwd.out["dx"], self.norm.h, self.nw, 1e-5, dh=self.dres)

    def run(self, stream=None):
        self.norm(stream)
        self.block(stream)
        st = torch.cuda.current_stream().cuda_stream if stream is None else stream
        fn = B.lib().moe_quant_act_mx if self.scheme == "mxfp8" else B.lib().moe_quant_act
        assert fn(self.block.h.data_ptr(), self.T, self.I, self.I, self.hq.data_ptr(), self.hs.data_ptr(), st) == 0
        self.down(stream)
        self.lora(stream)
        self.block_bwd(stream)
        self.norm_bwd(stream)

    def outs(self):
        b, n = self.block_bwd.out, self.norm_bwd.out
        return [self.norm.h, self.norm.y, self.norm.yq, self.norm.ys, self.block.h, self.block.gu, self.down.y,
                b["dgu"], b["dx"], b["dw"], b["dbias"], n["dx"], n["dweight"], n["dbias"]]


@pytest.mark.parametrize("scheme", ["fp8", "mxfp8"])
def test_dense_layer_and_its_gradients(scheme):
    c = _Layer(scheme)
    c.run()
    torch.cuda.synchronize()
    T, H, I = c.T, c.H, c.I
    h, y = OD.add_layernorm(c.xf, c.resf, c.nwf, c.nbf, 1e-5)
    assert np.array_equal(host(c.norm.h), h)
    within(host(c.norm.y), y, UB * np.abs(y) + 2.0 ** -28 * (np.abs(y) + np.abs(c.nbf)) + TINY, "norm")
    # the block on the codes that came out; matrix-core sums by the repository's accumulation model, eight of its
    # standard deviations
    q1, s1, q2, s2 = c.q
    micro = scheme == "mxfp8"
    xv, wv = OL.dequant_linear(c.norm.yq.cpu().numpy(), c.norm.ys.cpu().numpy(), q1, s1, micro)
    hh, g, u = OD.gated(xv, wv, c.b1f, "silu")
    err = 8 * omoe.ACC_ERR * np.sqrt((xv * xv) @ (wv * wv))
    gu = np.concatenate([g, u], 1)
    within(host(c.block.gu), gu, err + UB * (np.abs(gu) + err) + TINY, "gu")
    eg, eu = np.split(err, 2, axis=1)
    tol = 1.1 * eg * np.abs(u) + eu * np.abs(OD.activation(g, "silu")) + 1.1 * eg * eu + 32 * U * np.abs(hh) + 32 * U * np.abs(g * u)
    within(host(c.block.h), hh, tol + UB * (np.abs(hh) + tol) + TINY, "h")
    # down projection with the residual stream, rounded to bf16, then the adapters on top of it, rounded again
    hv, w2v = OL.dequant_linear(c.hq.cpu().numpy(), c.hs.cpu().numpy(), q2, s2, micro)
    base = hv @ w2v + h
    e2 = 8 * omoe.ACC_ERR * np.sqrt((hv * hv) @ (w2v * w2v))
    hb = host(c.block.h)
    yy, mag = OD.lora(hb, c.af, c.bf, c.sf, c.ids.tolist(), c.off.cpu().numpy(), base, base)
    tol = e2 + UB * (np.abs(base) + e2) + ((I + 64) * U + 2.0 ** -17) * mag
    within(host(c.down.y), yy, tol + UB * (np.abs(yy) + tol) + TINY, "y")
    # backward, from the values that the forward pass left
    guf = host(c.block.gu)
    v, m = OD.gated_backward(c.dhf, guf[:, :I], guf[:, I:], "silu")
    d = host(c.block_bwd.out["dgu"])
    within(d, v, UB * np.abs(v) + 256 * U * m + TINY, "dgu")
    for name, a, b, rounding in (("dx", d, wv.T, UB), ("dw", xv.T, d, 0.0)):
        ref, mg = a @ b, np.abs(a) @ np.abs(b)
        t = (a.shape[1] + 8) * U * mg
        within(host(c.block_bwd.out[name]), ref, t + rounding * (np.abs(ref) + t) + TINY, name)
    dx, dw, db, mg, wm, bm = OD.layernorm_backward(host(c.block_bwd.out["dx"]), h, c.nwf, 1e-5, c.dresf)
    within(host(c.norm_bwd.out["dx"]), dx, UB * np.abs(dx) + 10 * U * (1 + UB) * mg + TINY, "norm dx")
    within(host(c.norm_bwd.out["dweight"]), dw, (T + 48) * U * (wm + bm), "dweight")
    within(host(c.norm_bwd.out["dbias"]), db, (T + 48) * U * bm, "dbias")


def test_dense_layer_gradient_against_differences():
    """d/dx of sum(dh * block(norm(x))) by differences of the oracle, without the quantisation between."""
    T, H, I = 3, 128, 32
    g = rng(72)
    x, xf = bf16(g.standard_normal((T, H)))
    nw, nwf = f32(1 + 0.1 * g.standard_normal(H))
    nb, nbf = f32(0.1 * g.standard_normal(H))
    w = np.round(g.standard_normal((H, 2 * I)) * 4) / 32      # E4M3 values as they are
    lw = M.LinearWeights.from_float(torch.from_numpy(w.astype(np.float32)).to(DEV))
    dh, dhf = bf16(g.standard_normal((T, I)))
    n = M.moe_add_layernorm(x, nw, nb, 1e-5)
    gu = torch.from_numpy((host(n["y"]) @ w).astype(np.float32)).to(torch.bfloat16).to(DEV)
    b = M.moe_gated_linear_backward(dh, gu, lw, activation="silu")
    dx = host(M.moe_add_layernorm_backward(b["dx"], x, nw, 1e-5)["dx"])

    def loss(xx):
        return (OD.gated(OD.add_layernorm(xx, None, nwf, nbf, 1e-5)[1], w, None, "silu")[0] * dhf).sum(axis=1)
    step = 1e-5
    # y, gu, dgu and the block's dx are rounded to bf16 on the way: four times UB of the terms that make up a row
    _, gg, uu = OD.gated(OD.add_layernorm(xf, None, nwf, nbf, 1e-5)[1], w, None, "silu")
    _, m = OD.gated_backward(np.abs(dhf), np.abs(gg), np.abs(uu) + 1, "silu")
    size = (m + 1) @ np.abs(w).T
    r = 1 / np.sqrt(xf.var(axis=1, keepdims=True) + 1e-5)
    for _ in range(20):
        i, j = g.integers(T), g.integers(H)
        hi, lo = xf.copy(), xf.copy()
        hi[i, j] += step
        lo[i, j] -= step
        num = (loss(hi)[i] - loss(lo)[i]) / (2 * step)
        assert abs(dx[i, j] - num) <= 4 * UB * r[i, 0] * 2 * size[i].max() + 1e-4


def test_dense_layer_in_a_graph():
    """Captured once, replayed on new inputs in the same buffers (other adapters, other boundaries, padded rows) with
    eager calls of other objects between the replays."""
    c, other = _Layer("fp8"), _Layer("fp8", T=90, key=2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):      # nothing has run before the capture
            c.run()
    torch.cuda.synchronize()
    for rep in range(4):
        c.x.mul_(-0.75)
        c.dh.neg_()
        c.ids.copy_(torch.tensor([[0, 1, 2, 3, -1], [3, 9, 0, 0, 2], [1, 1, 1, 1, 1], [-1, -1, -1, -1, -1]][rep], dtype=torch.int32))
        c.off.copy_(torch.tensor([[0, 3, 3, 70, 100, 150], [5, 6, 7, 8, 9, 10], [0, 0, 0, 150, 150, 150], [0, 50, 60, 70, 80, 90]][rep],
                                 dtype=torch.int32))
        other.run()
        for o in c.outs():
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in c.outs()]
        for o in c.outs():
            o.zero_()
        c.run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, c.outs())):
            assert torch.equal(a, b), (rep, i)
    del graph


@pytest.mark.parametrize("T,K,I", [(5, 256, 64), (300, 384, 416), (1500, 2048, 352), (2300, 4096, 256), (9000, 256, 96)])
def test_gated_backward_variants_in_a_graph(T, K, I):
    """First call under capture, then replays against eager calls; sums in parts and not."""
    g = rng(73, T, K, I)
    gu, _ = bf16(g.standard_normal((T, 2 * I)))
    dh, _ = bf16(g.standard_normal((T, I)))
    x, _ = bf16(g.standard_normal((T, K)))
    xq, xs = M.moe_quant_act(x)
    w = M.LinearWeights.from_float(torch.randn(K, 2 * I, generator=torch.Generator().manual_seed(1)).to(DEV) * 0.05,
                                   bias=torch.zeros(2 * I, device=DEV))
    f = M.MoeGatedLinearBackward(dh, gu, w, xq, xs, dw_dtype=torch.bfloat16)
    e = M.MoeGatedLinearBackward(dh, gu, w, xq, xs, dw_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            f()
    for _ in range(3):
        dh.mul_(-1.25)
        for o in f.out.values():
            o.zero_()
        graph.replay()
        want = e()
        torch.cuda.synchronize()
        assert all(torch.equal(f.out[n], want[n]) for n in want)


def test_dense_layer_on_other_streams():
    c = _Layer("mxfp8")
    c.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in c.outs()]
    side = torch.cuda.Stream()
    for how in ("current", "explicit"):
        for o in c.outs():
            o.zero_()
        torch.cuda.synchronize()
        if how == "current":
            with torch.cuda.stream(side):
                c.run()
        else:
            c.run(side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.outs(), want)), how
    # two layers at once, an object per stream
    d = _Layer("mxfp8", key=3)
    d.run()
    torch.cuda.synchronize()
    want_d = [o.clone() for o in d.outs()]
    other = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            c.run()
        with torch.cuda.stream(other):
            d.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c.outs(), want)) and all(torch.equal(a, b) for a, b in zip(d.outs(), want_d))


def test_binding_refuses():
    c = _Layer("fp8")
    with pytest.raises(ValueError, match="activation"):
        M.MoeGatedLinear(c.norm.yq, c.norm.ys, c.w1, "tanh")
    with pytest.raises(ValueError, match="xs"):
        M.MoeGatedLinear(c.norm.yq, c.norm.ys[:, :2].contiguous(), c.w1)
    with pytest.raises(ValueError, match="dw needs"):
        M.MoeGatedLinearBackward(c.dh, c.block.gu, c.w1, want_dw=True)
    with pytest.raises(TypeError, match="dw_dtype"):
        M.MoeGatedLinearBackward(c.dh, c.block.gu, c.w1, dw_dtype=torch.float16)
    with pytest.raises(ValueError, match="gu"):
        M.MoeGatedLinearBackward(c.dh, c.dh, c.w1)
    with pytest.raises(TypeError, match="adapter_ids"):
        M.MoeLora(c.block.h, c.lw, c.ids.long(), c.off)
    with pytest.raises(ValueError, match="adapter_ids"):
        M.MoeLora(c.block.h, c.lw, c.ids)
    with pytest.raises(ValueError, match="seq_offsets"):
        M.MoeLora(c.block.h, c.lw, c.ids, c.off[:-1].contiguous())
    with pytest.raises(ValueError, match="b: expected"):
        M.MoeLora(c.block.h, M.LoraWeights(c.lw.a, c.lw.b[:, :, :8].contiguous()), c.ids, c.off)
    with pytest.raises(ValueError, match="bias"):
        M.MoeAddLayerNorm(c.x, c.nw, c.nb[:-8])
    with pytest.raises(TypeError, match="weight"):
        M.MoeAddLayerNorm(c.x, c.nw.double())
    with pytest.raises(B.MoeError, match="multiples of 8"):
        M.moe_lora(c.block.h, M.LoraWeights(c.lw.a[:, :4].contiguous(), c.lw.b[:, :, :4].contiguous()), c.ids, c.off)
    with pytest.raises(TypeError, match="GPU"):
        M.moe_lora(c.block.h, c.lw, c.ids.cpu(), c.off)
