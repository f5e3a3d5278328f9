"""Adapters of many requests on the GPU against the float64 oracle (oracle/dense.py); tolerances as in
test_gpu_layer.py."""
import numpy as np
import pytest
import torch

from oracle import dense as OD
from test_gpu_guards import Arena
from test_gpu_layer import TINY, U, UB, bf16, f32, host, rng, strided, within

pytestmark = pytest.mark.gpu

M = pytest.importorskip("mixture_experts_fp8_amd")
B = M.binding
DEV = "cuda"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _random_offsets(T, S, key, pad=0):
    g = rng(51, T, S, key)
    return np.concatenate([[0], np.sort(g.integers(0, T - pad + 1, S - 1)), [T - pad]]).tolist()


CASES = [  # T, K, N, R, adapters, sequences (None: one row each, a list: offsets, a number: random ones), out
    (1, 8, 16, 8, 1, None, "bf16"), (1, 7168, 2816, 16, 3, None, "bf16"), (32, 2816, 2816, 16, 24, None, "bf16"),
    (5, 72, 80, 24, 2, None, "f32"), (300, 136, 272, 8, 7, None, "bf16"), (7, 64, 48, 256, 4, None, "f32"),
    (9, 104, 64, 40, 3, [0, 0, 3, 3, 4, 9], "bf16"), (40, 768, 400, 64, 5, [2, 2, 20, 37, 37], "bf16"),
    (130, 1152, 144, 32, 4, [0, 1, 2, 3, 100, 129], "f32"), (65, 1032, 64, 72, 2, [0, 65], "bf16"),
    (500, 512, 528, 128, 3, [0, 64, 128, 500], "bf16"), (700, 256, 112, 256, 5, 9, "f32"), (1000, 640, 1040, 16, 6, 70, "bf16"),
    (2047, 1024, 512, 64, 12, 40, "bf16"), (5000, 64, 32, 16, 9, 4500, "bf16"), (3000, 128, 64, 48, 3, 3, "bf16"),
    (64, 4096, 256, 8, 2, [-5, 30, 90], "bf16"),     # offsets outside the rows
    (200, 448, 16, 200, 2, [150, 160, 190], "f32"), (4200, 320, 4112, 32, 4, 3, "bf16"),
    # windows of 32 rows at each rank's tiles and both types
    (2100, 136, 272, 24, 3, 5, "f32"), (2500, 520, 144, 64, 4, 60, "f32"), (2600, 320, 528, 16, 3, 20, "bf16"),
    (2050, 256, 64, 200, 2, [1000, 1990, 2049], "bf16"), (2200, 1096, 1040, 8, 5, 40, "f32"),
    # the largest depth, rank and width
    (3, 65536, 48, 256, 2, None, "f32"), (20, 65536, 16, 8, 2, [0, 3, 20], "bf16"), (2, 8, 1 << 20, 8, 2, None, "bf16"),
]


def _inputs(T, K, N, R, n, seqs, out, key=1, whole=False):
    g = rng(52, T, K, N, R, key)
    draw = (lambda lim, *s: g.integers(-lim, lim + 1, s).astype(np.float64)) if whole else (lambda lim, *s: g.standard_normal(s))
    x, xf = bf16(draw(3, T, K))
    a, af = bf16(draw(1, n, R, K) * (1 if whole else K ** -0.5))
    b, bf = bf16(draw(3, n, N, R) * (1 if whole else R ** -0.5))
    s, sf = f32(2.0 ** g.integers(-1, 2, n) if whole else 0.5 + g.random(n))
    r, rf = (bf16 if out == "bf16" else f32)(draw(9, T, N))
    off = None if seqs is None else seqs if isinstance(seqs, list) else _random_offsets(T, seqs, key)
    S = T if off is None else len(off) - 1
    ids = np.where(g.random(S) < 0.2, g.choice([-1, n, -2 ** 31, 2 ** 31 - 1], S), g.integers(0, n, S)).astype(np.int32)
    return x, xf, M.LoraWeights(a, b, s), (af, bf, sf), r, rf, ids, off


def _tolerance(K, R, mag, y, res, out):
    # inner sums of K terms and outer ones of R in parts, in any order; the parts' remainder; the scale's product
    t = ((K + 3 * R + 24) * U + (2.0 ** -17 if out == "bf16" else 2.0 ** -25)) * mag
    t = t + U * (np.abs(y) + np.abs(res))
    return t + (UB * (np.abs(y) + t) + TINY if out == "bf16" else 0)


@pytest.mark.parametrize("T,K,N,R,n,seqs,out", CASES)
def test_lora(T, K, N, R, n, seqs, out):
    print("lora", T, K, N, R, n, seqs if not isinstance(seqs, list) else len(seqs), out, flush=True)
    x, xf, w, (af, bf, sf), r, rf, ids, off = _inputs(T, K, N, R, n, seqs, out)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    idd, offd = _i32(ids), None if off is None else _i32(off)
    for residual in (True, False):
        res, resf = (r, rf) if residual else (None, None)
        y0 = torch.full((T, N), 7.0, dtype=dt, device=DEV)
        got = M.moe_lora(x, w, idd, offd, res, dt, y=y0)
        want, mag = OD.lora(xf, af, bf, sf, ids, off, resf, np.full((T, N), 7.0))
        within(host(got), want, np.where(mag > 0, _tolerance(K, R, mag, want, rf if residual else 0 * want, out), 0), "y")
        # without a scale: 1
        if residual:
            plain = M.moe_lora(x, M.LoraWeights(w.a, w.b), idd, offd, res, dt, y=torch.full_like(y0, 7.0))
            want1, mag1 = OD.lora(xf, af, bf, np.ones(n), ids, off, resf, np.full((T, N), 7.0))
            within(host(plain), want1, np.where(mag1 > 0, _tolerance(K, R, mag1, want1, rf, out), 0), "y without scale")
        # the same bits with strided rows and inside a wider matrix, and in place
        wide = torch.full((T, N + 24), 7.0, dtype=dt, device=DEV)
        again = M.moe_lora(strided(x, 16), w, idd, offd, strided(res, 8) if residual else None, dt, y=wide[:, 8:N + 8])
        assert torch.equal(again, got) and (wide[:, :8] == 7).all() and (wide[:, N + 8:] == 7).all()
        if residual:
            over = r.clone()
            M.moe_lora(x, w, idd, offd, over, dt, y=over)
            written = torch.zeros(T, dtype=torch.bool)
            for lo, hi in zip(*((range(T), range(1, T + 1)) if off is None else (np.clip(off[:-1], 0, T), np.clip(off[1:], 0, T)))):
                written[lo:hi] = True
            written = written.to(DEV)
            assert torch.equal(over[written], got[written]) and torch.equal(over[~written], r[~written])


@pytest.mark.parametrize("T,K,N,R,n,seqs,out", [(6, 200, 48, 16, 3, None, "f32"), (90, 328, 80, 72, 2, [0, 40, 41, 88], "f32"),
                                               (300, 640, 144, 128, 2, 3, "f32")])
def test_lora_exact(T, K, N, R, n, seqs, out):
    """Whole numbers: |v| <= 3 * 640 < 2^16, two bf16 values hold it; |y| <= 2^11 * 2 * 3 * 128 + 9 < 2^24."""
    x, xf, w, (af, bf, sf), r, rf, ids, off = _inputs(T, K, N, R, n, seqs, out, 2, whole=True)
    got = M.moe_lora(x, w, _i32(ids), None if off is None else _i32(off), r, torch.float32, y=torch.zeros_like(r))
    want, _ = OD.lora(xf, af, bf, sf, ids, off, rf, np.zeros((T, N)))
    assert np.array_equal(host(got), want)


def test_lora_rows_do_not_depend_on_the_batch():
    """A row's result is its own: other sequences hold infinities and NaN, also in rows and adapters that share a
    workgroup's tiles; rows outside the sequences are not read."""
    T, K, N, R, n = 100, 320, 144, 24, 4
    x, xf, w, _, r, rf, _, _ = _inputs(T, K, N, R, n, 4, "bf16", 3)
    off, ids = [5, 17, 50, 51, 90], [0, 1, 2, 3]
    want = M.moe_lora(x, w, _i32(ids), _i32(off), r)
    bad = x.clone()
    bad[:5], bad[17:50], bad[90:] = float("nan"), float("inf"), float("nan")
    a = w.a.clone()
    a[1], a[3, :, 7] = float("nan"), float("inf")
    got = M.moe_lora(bad, M.LoraWeights(a, w.b, w.scale), _i32(ids), _i32(off), r)
    for rows in (slice(0, 17), slice(50, 51), slice(90, 100)):
        assert torch.equal(got[rows], want[rows])
    assert torch.isnan(got[17:50]).all() and not torch.isfinite(got[51:90].float()).any()
    # the same rows as a batch of their own
    one = M.moe_lora(x[51:90].contiguous(), w, _i32([3]), _i32([0, 39]), r[51:90].contiguous())
    assert torch.equal(one, want[51:90])


def test_lora_in_the_columns_of_one_matrix():
    """Projections side by side in the rows of one matrix, each with adapters of its own, in place."""
    T, K, R, n = 70, 256, 16, 3
    x, _, _, _, _, _, _, _ = _inputs(T, K, 16, R, n, None, "bf16", 4)
    y = bf16(rng(53).standard_normal((T, 208)))[0]
    ids = _i32(rng(54).integers(-1, n, T))
    before = y.clone()
    for lo, hi in ((0, 64), (64, 192)):
        _, _, w, _, _, _, _, _ = _inputs(T, K, hi - lo, R, n, None, "bf16", 5)
        alone = M.moe_lora(x, w, ids, residual=before[:, lo:hi].contiguous())
        M.moe_lora(x, w, ids, residual=y[:, lo:hi], y=y[:, lo:hi])
        assert torch.equal(y[:, lo:hi], alone)
    assert torch.equal(y[:, 192:], before[:, 192:])


@pytest.mark.parametrize("T,K,N,R,n,seqs,out", [(7, 2816, 208, 16, 3, None, "bf16"), (130, 520, 144, 72, 4, [0, 1, 64, 127], "f32"),
                                               (900, 256, 272, 32, 2, 4, "bf16")])
def test_lora_stays_inside_its_buffers(T, K, N, R, n, seqs, out):
    x, _, w, _, r, _, ids, off = _inputs(T, K, N, R, n, seqs, out, 6)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    args = (x, w, _i32(ids), None if off is None else _i32(off), r, dt)
    want = M.moe_lora(*args, y=torch.zeros_like(r))
    need = B.lib().moe_lora_workspace_size(T, R, len(ids), int(off is not None), int(out == "bf16"))
    ar = Arena([T * N * r.element_size(), need])
    call = M.MoeLora(*args)
    ar.view(0, dt, (T, N)).zero_()
    call.args.y, call.args.workspace, call.args.workspace_bytes = ar.ptr(0), ar.ptr(1), need
    call()
    ar.assert_guards("lora")
    assert torch.equal(ar.view(0, dt, (T, N)), want)
