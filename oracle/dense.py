"""The operators of dense layers (CPU, float64): residual + layer norm, gated feed-forward block,
adapters of many requests, and the gradients of the first two.

TEST INFRASTRUCTURE ONLY: nothing in the product path may import this module.

Definitions as stated in include/moe_fp8.h.  Pins (tests/test_oracle_dense.py): the gradients agree
with central differences of the forward functions here; closed forms and hand values.
"""
from __future__ import annotations

import numpy as np

from .layer import activation
from .w8a16 import bf16_rne


# ---- residual + layer norm ---------------------------------------------------------------
def _standard(h, eps):
    d = h - h.mean(axis=1, keepdims=True)
    return d, 1.0 / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)


def add_layernorm(x, residual, weight, bias, eps):
    """(h, y) float64: h rounded to bf16, y not rounded."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = bf16_rne(h + residual)
    d, r = _standard(h, eps)
    y = d * r * weight
    return h, y if bias is None else y + bias


def layernorm_backward(dy, h, weight, eps, dh=None):
    """(dx, dweight, dbias, dx_mag, dweight_mag, dbias_mag): the gradients and the sums of the absolute
    values of the terms that they are made of."""
    H = h.shape[1]
    d, r = _standard(h, eps)
    xh, g = d * r, dy * weight
    dx = r * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    mag = r * (np.abs(g) + np.abs(g).mean(axis=1, keepdims=True) + np.abs(xh) * np.abs(g * xh).sum(axis=1, keepdims=True) / H)
    if dh is not None:
        dx, mag = dx + dh, mag + np.abs(dh)
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0), mag, np.abs(dy * xh).sum(axis=0), np.abs(dy).sum(axis=0)


# ---- gated feed-forward block ------------------------------------------------------------
def gated(x, w, bias=None, act="silu"):
    """(h, g, u) from the operands' values; w: gate columns, then up columns."""
    v = x @ w
    if bias is not None:
        v = v + bias
    g, u = np.split(v, 2, axis=1)
    return activation(g, act) * u, g, u
