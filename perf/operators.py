"""Operators that stand around the routed expert step, as measured cases.

* norm:    residual addition + RMS norm with E4M3 codes and UE8M0 scales (the input of the
           expert step and of the FP8 projections), and its backward pass;
* linear:  FP8 matrix product with bias, activation and residual in its epilogue;
* balance: load-balance and z losses with per-expert counts, and the router's gradient;
* combine: backward pass of the weighted top-k combine.

`run` gives either the plain form (elementary torch operations in 32 bits) or, where `own` is
true, the calls of the library.  `exact` restates each definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---- cases ------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the 128-expert gate: 32 sequences, a token each; latency counts
        dict(name="norm_decode", op="norm", T=32, H=2816, group=128, residual=True, backward=False),
        # the input of a prefill's expert step with one scale per 32 columns
        dict(name="norm_prefill_mx", op="norm", T=4096, H=7168, group=32, residual=True, backward=False),
        # the norm's gradients in a training step over a large batch
        dict(name="norm_gradient", op="norm", T=16384, H=4096, group=0, residual=True, backward=True),
        # a single token through an attention output projection: the weights are streamed once
        dict(name="linear_token", op="linear", T=1, K=7168, N=7168, mx=False, act="none", bias=False, residual=True),
        # a decode batch through a biased projection with one scale per 32 elements
        dict(name="linear_decode_mx", op="linear", T=32, K=2816, N=2816, mx=True, act="gelu", bias=True, residual=False),
        # a ragged batch through a short dense layer
        dict(name="linear_unaligned", op="linear", T=2047, K=768, N=2304, mx=False, act="silu", bias=True, residual=False),
        # a large prefill through a square projection added to the residual stream
        dict(name="linear_prefill", op="linear", T=16384, K=4096, N=4096, mx=False, act="none", bias=False, residual=True),
        # the smallest router: losses and gradient of 64 tokens over 8 experts
        dict(name="balance_tiny", op="balance", T=64, E=8, k=2, scoring="softmax", renorm=True, seqs=1, pad=0, skew=0.0),
        # packed sequences of uneven lengths with padding behind the last, sigmoid scores
        dict(name="balance_sequences", op="balance", T=4096, E=256, k=8, scoring="sigmoid", renorm=True, seqs=9, pad=37, skew=0.5),
        # one large batch whose experts are unevenly loaded
        dict(name="balance_prefill", op="balance", T=16384, E=128, k=8, scoring="softmax", renorm=False, seqs=1, pad=0, skew=1.5),
        # routing-weight gradients of frozen experts, float32 expert outputs
        dict(name="combine_weights", op="combine", T=2047, H=768, E=256, k=8, bf16=False, d_out=False),
        # the whole gradient of the combine of a large batch, bf16 expert outputs
        dict(name="combine_gradient", op="combine", T=16384, H=4096, E=128, k=8, bf16=True, d_out=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "linear", "balance", "combine"))
    if op == "norm":
        backward = rng.random() < 0.4
        group = 0 if backward else rng.choice((0, 32, 128))
        step = group or 8
        H = step * _log_int(rng, max(1, 64 // step), 8192 // step)
        T = _log_int(rng, 1, min(16384, 16384 * 4096 // H))
        return dict(op=op, T=T, H=H, group=group, residual=rng.random() < 0.7, backward=backward)
    if op == "linear":
        K = 128 * _log_int(rng, 1, 64)
        N = 128 * _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(16384, 16384 * 4096 * 4096 // (K * N))))
        return dict(op=op, T=T, K=K, N=N, mx=rng.random() < 0.4, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    if op == "balance":
        E = _log_int(rng, 4, 512)
        T = _log_int(rng, 1, min(16384, 16384 * 128 // E))
        pad = rng.choice((0, 0, T // 9))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), scoring=rng.choice(("softmax", "sigmoid")),
                    renorm=rng.random() < 0.5, seqs=_log_int(rng, 1, 48), pad=pad, skew=rng.choice((0.0, 0.5, 1.5)))
    H = 8 * _log_int(rng, 8, 1024)
    E = _log_int(rng, 8, 256)
    k = rng.randint(1, 8)
    T = _log_int(rng, 1, min(16384, 16384 * 8 * 4096 // (H * k * 2)))
    return dict(op=op, T=T, H=H, E=E, k=k, bf16=rng.random() < 0.5, d_out=rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _hidden(g, T, H):
    """Residual-stream values: unit normal with a few large channels."""
    ch = torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 12.0, 1.0)
    return (_randn(g, T, H) * ch).to(torch.bfloat16)


def _exponent(amax, largest):
    """The smallest integer e in [-127, 127] with amax <= largest * 2^e; 0 where amax is 0."""
    m, x = torch.frexp(amax / largest)          # amax / largest = m 2^x, m in [0.5, 1)
    e = torch.where(m == 0.5, x - 1, x)
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(-127, 127))


def _codes(v, e):
    """E4M3 codes of v / 2^e, bytes."""
    return torch.ldexp(v, -e).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(q):
    return q.view(torch.float8_e4m3fn).float()


def _pow2(s, dtype=torch.float32):
    """2^(s - 127) of UE8M0 bytes."""
    return torch.exp2(s.to(dtype) - 127)


def _router(g, T, E, k, skew):
    logits = _randn(g, T, E) + skew * _randn(g, E)
    return logits, torch.topk(logits, k, dim=1).indices.to(torch.int32)


def _inputs(c, seed):
    g, s = _gen(seed), {"case": c}
    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        s["weight"] = 1 + 0.1 * _randn(g, H)
        s["x"] = _hidden(g, T, H)
        if c["backward"]:   # x: the normalised row's input h; dy: the gradient that arrives
            s["dy"] = (0.01 * _randn(g, T, H)).to(torch.bfloat16)
            s["dres"] = (0.01 * _randn(g, T, H)).to(torch.bfloat16) if c["residual"] else None
        else:
            s["residual"] = _hidden(g, T, H) if c["residual"] else None
    elif c["op"] == "linear":
        K, N = c["K"], c["N"]
        x, w = _hidden(g, T, K).float(), 0.02 * _randn(g, K, N)
        gs = 32 if c["mx"] else 128
        e = _exponent(x.view(T, K // gs, gs).abs().amax(-1), 448.0)
        s["xq"], s["xs"] = _codes(x, e.repeat_interleave(gs, 1)), (e + 127).to(torch.uint8)
        if c["mx"]:         # one scale per 32 rows of K and one column
            e = _exponent(w.view(K // 32, 32, N).abs().amax(1), 448.0)
            s["wq"], s["ws"] = _codes(w, e.repeat_interleave(32, 0)), (e + 127).to(torch.uint8)
        else:               # one scale per 128 x 128 block
            e = _exponent(w.view(K // 128, 128, N // 128, 128).abs().amax((1, 3)), 448.0)
            s["wq"] = _codes(w, e.repeat_interleave(128, 0).repeat_interleave(128, 1))
            s["ws"] = (e + 127).to(torch.uint8)
        s["bias"] = 0.1 * _randn(g, N) if c["bias"] else None
        s["residual"] = _hidden(g, T, N) if c["residual"] else None
    elif c["op"] == "balance":
        s["logits"], s["ids"] = _router(g, T, c["E"], c["k"], c["skew"])
        s["dweights"] = 0.01 * _randn(g, T, c["k"])
        n = T - c["pad"]    # sequence boundaries, empty sequences among them by chance
        cuts = torch.randint(0, n + 1, (c["seqs"] - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, n], device="cuda")
        s["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        s["whole"] = c["seqs"] == 1 and c["pad"] == 0
        s["coef"] = (1e-2, 1e-3)
    else:
        H, k = c["H"], c["k"]
        _, ids = _router(g, T, max(c["E"], k), k, 0.5)
        order = torch.sort(ids.reshape(-1), stable=True).indices
        pos = torch.empty_like(order)
        pos[order] = torch.arange(T * k, device="cuda")
        s["pos"] = pos.to(torch.int32)
        s["weights"] = torch.softmax(_randn(g, T, k), 1)
        s["eo"] = _randn(g, T * k, H).to(torch.bfloat16) if c["bf16"] else _randn(g, T * k, H)
        s["dy"] = (0.01 * _randn(g, T, H)).to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:     # the handle and the packed weights that a program keeps
        import mixture_experts_fp8_amd as M
        c = case
        if c["op"] == "norm":
            if c["backward"]:
                s["call"] = M.MoeAddRmsNormBackward(s["dy"], s["x"], s["weight"], EPS, dh=s["dres"])
            else:
                quant = {0: None, 32: M.MOE_QUANT_MXFP8, 128: M.MOE_QUANT_FP8_BLOCK128}[c["group"]]
                s["call"] = M.MoeAddRmsNorm(s["x"], s["weight"], EPS, residual=s["residual"], quant=quant)
                if quant is not None:   # the output buffers under the types that their bytes stand for
                    s["named"] = _named_codes(s["call"].yq, s["call"].ys)
        elif c["op"] == "linear":
            w = M.LinearWeights.from_logical(s["wq"], s["ws"], M.MOE_QUANT_MXFP8 if c["mx"] else M.MOE_QUANT_FP8_BLOCK128,
                                             bias=s["bias"])
            s["call"] = M.MoeLinear(s["xq"], s["xs"], w, activation=c["act"], residual=s["residual"])
        elif c["op"] == "balance":
            p = M.route_params(c["E"], c["k"], c["scoring"], c["renorm"])
            offsets = None if s["whole"] else s["offsets"]
            a, b = s["coef"]
            s["loss"] = M.MoeBalanceLoss(p, s["logits"], s["ids"], seq_offsets=offsets, balance_coef=a, z_coef=b)
            s["call"] = M.MoeRouteBackward(p, s["logits"], s["ids"], dweights=s["dweights"], counts=s["loss"].counts,
                                           seq_offsets=offsets, balance_coef=a, z_coef=b)
        else:
            s["call"] = M.MoeCombineBackward(s["dy"], s["eo"], s["pos"], s["weights"], d_expert_out=c["d_out"])
    return s


# ---- one pass ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"norm": _norm, "linear": _linear, "balance": _balance, "combine": _combine}[c["op"]](c, state)


def _named_codes(q, s):
    """Codes as the E4M3 values and scales as the powers of two that they stand for."""
    return {"yq": q.view(torch.float8_e4m3fn), "ys": s.view(torch.float8_e8m0fnu)}


def _own(c, s):
    if c["op"] == "norm":
        r = s["call"]()
        if c["backward"]:
            return {"dx": r["dx"], "dweight": r["dweight"]}
        out = {"y": r["y"]}
        if c["residual"]:
            out["h"] = r["h"]
        if c["group"]:
            out.update(s["named"])
        return out
    if c["op"] == "linear":
        return {"y": s["call"]()}
    if c["op"] == "balance":
        r = s["loss"]()
        return {"losses": r["losses"], "counts": r["counts"], "mean_probs": r["mean_probs"], "dlogits": s["call"]()}
    r = s["call"]()
    return {n: r[n] for n in (("dweights", "d_expert_out") if c["d_out"] else ("dweights",))}


def _norm(c, s):
    w = s["weight"]
    if c["backward"]:
        h, dy = s["x"].float(), s["dy"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        xh, gw = h * r, dy * w
        dx = r * (gw - xh * (gw * xh).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xh).sum(0)}
    out, h = {}, s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
        out["h"] = h
    f = h.float()
    y = (f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * w).to(torch.bfloat16)
    out["y"] = y
    if c["group"]:
        v, gs = y.float(), c["group"]
        e = _exponent(v.view(c["T"], c["H"] // gs, gs).abs().amax(-1), 448.0)
        out.update(_named_codes(_codes(v, e.repeat_interleave(gs, 1)), (e + 127).to(torch.uint8)))
    return out


def _act(v, name):
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _linear(c, s):
    gs = 32 if c["mx"] else 128
    x = _value(s["xq"]) * _pow2(s["xs"]).repeat_interleave(gs, 1)
    ws = _pow2(s["ws"]).repeat_interleave(gs, 0)
    w = _value(s["wq"]) * (ws if c["mx"] else ws.repeat_interleave(128, 1))
    v = x @ w
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _act(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return {"y": v.to(torch.bfloat16)}


def _balance(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    l, off = s["logits"], s["offsets"].long()
    t = torch.arange(T, device=l.device)
    member = ((t >= off[:-1, None]) & (t < off[1:, None])).float()            # [S, T]
    inside = (t >= off[0]) & (t < off[-1])
    hit = (s["ids"].long()[:, :, None] == torch.arange(E, device=l.device))   # [T, k, E]
    n = member.sum(1, keepdim=True)                                           # tokens per sequence
    counts = member @ hit.float().sum(1)
    lse = torch.logsumexp(l, 1)
    sig = 1 / (1 + torch.exp(-l))
    softmax = c["scoring"] == "softmax"
    p = torch.exp(l - lse[:, None]) if softmax else sig / sig.sum(1, keepdim=True)
    mean_p = (member @ p) / n.clamp(min=1)
    live, valid = (n > 0).sum().clamp(min=1), n.sum().clamp(min=1)
    a, b = s["coef"]
    frac = counts * (E / k) / n.clamp(min=1)                                  # load of each expert
    bal = a * (frac * mean_p).sum() / live
    z = b * torch.where(inside, lse * lse, 0).sum() / valid
    # gradient of the losses
    u = member.t() @ (a / live * frac / n.clamp(min=1))                       # dL/dp of each token
    d = p * (u - (p * u).sum(1, keepdim=True)) * (1 if softmax else 1 - sig)
    d = d + 2 * b / valid * (lse * inside)[:, None] * torch.exp(l - lse[:, None])
    # gradient through the routing weights
    dw = (hit * s["dweights"][:, :, None]).sum(1)
    if softmax and not c["renorm"]:
        g = p * (dw - (p * dw).sum(1, keepdim=True))
    else:
        score = p if softmax else sig
        q = torch.where(hit.any(1), score, 0)
        q = q / q.sum(1, keepdim=True)
        g = q * (dw - (q * dw).sum(1, keepdim=True)) * (1 if softmax else 1 - sig)
    d = (d + g) * inside[:, None]
    return {"losses": torch.stack([bal + z, bal, z]), "counts": counts.to(torch.int32), "mean_probs": mean_p, "dlogits": d}


def _combine(c, s):
    T, H, k = c["T"], c["H"], c["k"]
    pos, dy = s["pos"].long(), s["dy"].float()
    rows = s["eo"][pos].float().view(T, k, H)
    out = {"dweights": (rows * dy[:, None, :]).sum(2)}
    if c["d_out"]:
        d = torch.empty_like(s["eo"])
        d[pos] = (s["weights"][:, :, None] * dy[:, None, :]).view(T * k, H).to(d.dtype)
        out["d_expert_out"] = d
    return out


# ---- what one pass cannot do without ----------------------------------------------------
def work(c):
    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        n = T * H
        if c["backward"]:
            return dict(bytes=n * 2 * (3 + c["residual"]) + 8 * H, flops=12 * n)
        return dict(bytes=n * 2 * (2 + 2 * c["residual"]) + (n + n // c["group"] if c["group"] else 0) + 4 * H, flops=6 * n)
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        scales = (T * K + K * N) // 32 if c["mx"] else T * K // 128 + K * N // 16384
        return dict(bytes=T * K + K * N + scales + 2 * T * N * (1 + c["residual"]) + 4 * N * c["bias"], flops=2 * T * K * N)
    if c["op"] == "balance":
        E, k = c["E"], c["k"]
        return dict(bytes=T * E * 8 + T * k * 8 + c["seqs"] * E * 8, flops=16 * T * E)
    H, k = c["H"], c["k"]
    size = 2 if c["bf16"] else 4
    return dict(bytes=T * k * H * size * (1 + c["d_out"]) + T * H * 2 + T * k * (4 + 4 + 4 * c["d_out"]),
                flops=T * k * H * (2 + c["d_out"]))


# ---- the definitions in 64 bits ---------------------------------------------------------
def _round64(v, bits, low):
    """v to the nearest of the floats with `bits` significant bits whose smallest step is 2^low, ties to even."""
    _, x = torch.frexp(v)
    step = torch.exp2((x - bits).clamp(min=low).double())
    return torch.round(v / step) * step


def exact(case, seed):
    s, c = _inputs(case, seed), case
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "linear":
        return _exact_linear(c, s)
    if c["op"] == "balance":
        return _exact_balance(c, s)
    return _exact_combine(c, s)


def _exact_norm(c, s):
    H, w = c["H"], s["weight"].double()
    if c["backward"]:
        h, g = s["x"].double(), s["dy"].double()
        ms = h.square().sum(1, keepdim=True) / H + EPS
        # d/dh of g . (w h / sqrt(ms)) = g w / sqrt(ms) - h (g . w h) / (H ms^1.5)
        dot = (g * w * h).sum(1, keepdim=True)
        dx = g * w / ms.sqrt() - h * dot / (H * ms * ms.sqrt())
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dweight": (g * h / ms.sqrt()).sum(0)}
    out = {}
    h = s["x"].double()
    if s["residual"] is not None:
        h = _round64(h + s["residual"].double(), 8, -133)
        out["h"] = h
    y = _round64(h / (h.square().sum(1, keepdim=True) / H + EPS).sqrt() * w, 8, -133)
    out["y"] = y
    if c["group"]:
        grp = y.view(c["T"], -1, c["group"])
        top = grp.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top == 0, 448.0, top) / 448.0) - 1e-12).clamp(-127, 127)
        out["yq"] = _round64(grp * torch.exp2(-e), 4, -9).view(c["T"], H)
        out["ys"] = torch.exp2(e).squeeze(2)
    return out


def _exact_linear(c, s):
    T, K, N = c["T"], c["K"], c["N"]

    def decode(b):      # sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities
        b = b.to(torch.int32)
        ex, m = (b >> 3) & 15, (b & 7).double()
        mag = torch.where(ex == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((ex - 10).double()))
        return torch.where(b > 127, -mag, mag)

    per = 32 if c["mx"] else 128
    x = (decode(s["xq"]).view(T, K // per, per) * _pow2(s["xs"], torch.float64)[:, :, None]).view(T, K)
    ws = _pow2(s["ws"], torch.float64)
    if c["mx"]:
        w = (decode(s["wq"]).view(K // 32, 32, N) * ws[:, None, :]).view(K, N)
    else:
        w = (decode(s["wq"]).view(K // 128, 128, N // 128, 128) * ws[:, None, :, None]).view(K, N)
    v = torch.matmul(x, w)
    del x, w
    if s["bias"] is not None:
        v += s["bias"].double()
    if c["act"] == "relu":
        v = torch.where(v > 0, v, 0.0)
    elif c["act"] == "silu":
        v = v * torch.special.expit(v)
    elif c["act"] == "gelu":
        v = v * torch.special.erfc(-v / 2 ** 0.5) / 2
    elif c["act"] == "gelu_tanh":   # 1 + tanh(t) = 2 expit(2 t)
        v = v * torch.special.expit(2 * (2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    if s["residual"] is not None:
        v += s["residual"].double()
    return {"y": v}


def _exact_balance(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    l, ids = s["logits"].double().requires_grad_(), s["ids"].long()
    off = s["offsets"].tolist()
    a, b = s["coef"]
    prob = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
    if c["scoring"] == "sigmoid":
        prob = prob / prob.sum(1, keepdim=True)
    lens = [hi - lo for lo, hi in zip(off, off[1:])]
    live, valid = max(1, sum(n > 0 for n in lens)), max(1, sum(lens))
    bal = torch.zeros((), dtype=torch.float64, device=l.device)
    counts, means = [], []
    for lo, hi in zip(off, off[1:]):
        n = torch.bincount(ids[lo:hi].reshape(-1), minlength=E)
        counts.append(n)
        if hi > lo:
            means.append(prob[lo:hi].mean(0))
            bal = bal + (E / (k * (hi - lo)) * n * means[-1]).sum() * (a / live)
        else:
            means.append(torch.zeros(E, dtype=torch.float64, device=l.device))
    z = torch.logsumexp(l[off[0]:off[-1]], 1).square().sum() * (b / valid)
    sel = torch.gather(torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l), 1, ids)
    if c["scoring"] == "sigmoid" or c["renorm"]:
        sel = sel / sel.sum(1, keepdim=True)
    through = (sel * s["dweights"].double())[off[0]:off[-1]].sum()
    (d,) = torch.autograd.grad(bal + z + through, l)
    bal, z = bal.detach(), z.detach()
    return {"losses": torch.stack([bal + z, bal, z]), "counts": torch.stack(counts).to(torch.int32),
            "mean_probs": torch.stack(means).detach(), "dlogits": d}


def _exact_combine(c, s):
    T, H, k = c["T"], c["H"], c["k"]
    dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
    d = torch.empty(T * k, H, dtype=torch.float64, device="cuda") if c["d_out"] else None
    pos = s["pos"].view(T, k).long()
    dy = s["dy"].double()
    for j in range(k):
        dw[:, j] = (s["eo"].index_select(0, pos[:, j]).double() * dy).sum(1)
        if d is not None:
            d.index_copy_(0, pos[:, j], dy * s["weights"][:, j:j + 1].double())
    return {"dweights": dw, "d_expert_out": d} if d is not None else {"dweights": dw}
