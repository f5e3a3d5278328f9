"""Operators of dense layers on buffers whose offsets pass 2^31 elements or bytes, against the same rows alone and
against sums in 64 bits."""
import numpy as np
import pytest
import torch

from test_gpu_layer import bf16, rng

pytestmark = pytest.mark.gpu

M = pytest.importorskip("mixture_experts_fp8_amd")
DEV = "cuda"


def _free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_lora_rows_far_apart():
    """x and y 2^17 elements from row to row: 20000 rows are 5.2 GB each."""
    T, K, N, R, ld = 20000, 136, 48, 16, 1 << 17
    g = rng(81)
    x, _ = bf16(g.standard_normal((T, K)))
    r, _ = bf16(g.standard_normal((T, N)))
    w = M.LoraWeights(bf16(g.standard_normal((3, R, K)) * 0.1)[0], bf16(g.standard_normal((3, N, R)) * 0.1)[0])
    off = torch.tensor([0, 7000, 7001, T], dtype=torch.int32, device=DEV)
    ids = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    want = M.moe_lora(x, w, ids, off, r)
    xw = torch.empty(T, ld, dtype=torch.bfloat16, device=DEV)
    yw = torch.empty(T, ld, dtype=torch.bfloat16, device=DEV)
    xw[:, 1024:1024 + K] = x
    yw[:, :N] = r
    M.moe_lora(xw[:, 1024:1024 + K], w, ids, off, yw[:, :N], y=yw[:, :N])
    assert torch.equal(yw[:, :N], want)
    del xw, yw
    _free()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_lora_of_very_many_sequences(dt):
    """2^20 sequences, nearly all of them empty: slots of several launches, two rounds of the search more."""
    T, S, K, N, R, n = 300, 1 << 20, 72, 4624, 24, 5
    g = rng(82)
    x, _ = bf16(g.standard_normal((T, K)))
    r = bf16(g.standard_normal((T, N)))[0].to(dt)
    w = M.LoraWeights(bf16(g.standard_normal((n, R, K)) * 0.1)[0], bf16(g.standard_normal((n, N, R)) * 0.1)[0])
    at = np.sort(np.concatenate([[0, 1, 63, 64, S - 1], g.choice(np.arange(65, S - 1), 20, replace=False)]))   # the others: empty
    ends = np.concatenate([np.sort(g.choice(np.arange(4, T - 8), 24, replace=False)), [T - 5]])
    off = np.full(S + 1, 3, np.int32)
    for s, e in zip(at, ends):
        off[s + 1:] = e
    ids = g.integers(0, n, S).astype(np.int32)
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device=DEV)   # noqa: E731
    want = M.moe_lora(x, w, i32(ids[at]), i32(np.concatenate([[3], ends])), r, dt, y=torch.full_like(r, 7))
    got = M.moe_lora(x, w, i32(ids), i32(off), r, dt, y=torch.full_like(r, 7))
    assert torch.equal(got, want) and (got[:3] == 7).all() and (got[T - 5:] == 7).all() and (got[3:T - 5] != 7).any(1).all()
    _free()


def test_gated_linear_past_2_to_31_sums():
    """70000 x 2 x 16384 sums: 4.6 GB."""
    T, K, I = 70000, 128, 16384
    xq = torch.randint(0, 119, (T, K), dtype=torch.uint8, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    xs = torch.full((T, 1), 122, dtype=torch.uint8, device=DEV)
    w = M.LinearWeights.from_float(torch.randn(K, 2 * I, device=DEV, generator=torch.Generator(DEV).manual_seed(2)) * 0.1)
    out = M.moe_gated_linear(xq, xs, w, "silu", want_gu=True)
    for rows in (slice(0, 40), slice(65500, 65600), slice(T - 70, T)):
        part = M.moe_gated_linear(xq[rows].contiguous(), xs[rows].contiguous(), w, "silu", want_gu=True)
        assert torch.equal(part["h"], out["h"][rows]) and torch.equal(part["gu"], out["gu"][rows])
    del out, part
    _free()


def test_gated_linear_backward_near_its_limit():
    """33000 x 2 x 16224, just below 2^30 sums with the rows rounded up: operands of 2 GB."""
    T, K, I = 33000, 128, 16224
    gen = torch.Generator(DEV).manual_seed(3)
    gu = torch.randint(-2, 3, (T, 2 * I), device=DEV, generator=gen, dtype=torch.int8).to(torch.bfloat16)
    dh = torch.randint(-1, 2, (T, I), device=DEV, generator=gen, dtype=torch.int8).to(torch.bfloat16)
    xq = torch.randint(0, 2, (T, K), device=DEV, generator=gen, dtype=torch.int32).mul_(0x38).to(torch.uint8)    # 0 and 1
    xs = torch.full((T, 1), 127, dtype=torch.uint8, device=DEV)
    wv = torch.randint(-1, 2, (K, 2 * I), device=DEV, generator=gen, dtype=torch.int32).float()
    w = M.LinearWeights.from_float(wv)
    out = M.moe_gated_linear_backward(dh, gu, w, xq, xs, "none", want_dbias=True)
    x = (xq != 0).double()
    for c in (slice(0, 48), slice(I - 64, I)):      # whole numbers below 2^24: exact
        dg, du = dh[:, c].double() * gu[:, I:][:, c].double(), dh[:, c].double() * gu[:, :I][:, c].double()
        assert torch.equal(out["dgu"][:, c].double(), dg) and torch.equal(out["dgu"][:, I:][:, c].double(), du)
        assert torch.equal(out["dw"][:, c].double(), x.t() @ dg) and torch.equal(out["dw"][:, I:][:, c].double(), x.t() @ du)
        assert torch.equal(out["dbias"][c].double(), dg.sum(0)) and torch.equal(out["dbias"][I:][c].double(), du.sum(0))
    for r in (slice(0, 64), slice(T - 70, T)):
        ref = out["dgu"][r].double() @ wv.double().t()
        assert torch.equal(out["dx"][r], ref.to(torch.bfloat16))
    with pytest.raises(M.MoeError, match="2\\^30"):
        e = torch.empty(33100, 2 * I, dtype=torch.bfloat16, device=DEV)
        M.MoeGatedLinearBackward(e[:, :I].contiguous(), e, w, want_dx=False)()
    del out, gu, dh
    _free()


def test_add_layernorm_past_2_to_31_elements():
    T, H = 300000, 8192
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(DEV).manual_seed(4))
    w, b = torch.rand(H, device=DEV), torch.rand(H, device=DEV)
    y = M.moe_add_layernorm(x, w, b, quant=M.MOE_QUANT_FP8_BLOCK128)
    rows = slice(T - 50, T)
    part = M.moe_add_layernorm(x[rows].contiguous(), w, b, quant=M.MOE_QUANT_FP8_BLOCK128)
    for n in ("y", "yq", "ys"):
        assert torch.equal(part[n], y[n][rows])
    d = M.moe_add_layernorm_backward(y["y"], x, w, want_dweight=False, want_dbias=False)["dx"]
    assert torch.equal(d[rows], M.moe_add_layernorm_backward(y["y"][rows], x[rows], w)["dx"])
    del x, y, d
    _free()
