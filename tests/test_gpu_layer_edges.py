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
