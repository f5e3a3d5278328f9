"""The operators of dense layers (CPU, float64): residual + layer norm, gated feed-forward block,
adapters of many requests, and the gradients of the first two.

TEST INFRASTRUCTURE ONLY: nothing in the product path may import this module.

Definitions as stated in include/moe_fp8.h.  Pins (tests/test_oracle_dense.py): the gradients agree
with central differences of the forward functions here; closed forms and hand values.
"""
from __future__ import annotations

import math

import numpy as np

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
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _factor(v, name):
    """(p, q, slope of the logistic's argument): the activation is v p, and q = 1 - p.  1 + tanh(t) is formed as
    2 / (1 + exp(-2 t)) and 1 + erf(t) as erfc(-t): their sums lose every digit far below 0."""
    with np.errstate(over="ignore"):
        if name == "silu":
            return 1.0 / (1.0 + np.exp(-v)), 1.0 / (1.0 + np.exp(v)), np.ones_like(v)
        c = 2.0 * math.sqrt(2.0 / math.pi)
        t = c * (v + 0.044715 * v ** 3)
        return 1.0 / (1.0 + np.exp(-t)), 1.0 / (1.0 + np.exp(t)), c * (1.0 + 3 * 0.044715 * v * v)


def activation(v, name):
    v = np.asarray(v, dtype=np.float64)
    if name == "none":
        return v
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    if name in ("silu", "gelu_tanh"):
        return v * _factor(v, name)[0]
    raise ValueError(name)


def activation_slope(v, name):
    """(slope, sum of the absolute values of its terms)."""
    v = np.asarray(v, dtype=np.float64)
    if name == "none":
        return np.ones_like(v), np.ones_like(v)
    if name == "relu":
        return (v > 0).astype(np.float64), np.ones_like(v)
    if name == "gelu":
        p, b = 0.5 * _erfc(-v / math.sqrt(2.0)), v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    elif name in ("silu", "gelu_tanh"):
        p, q, s = _factor(v, name)
        b = v * p * q * s
    else:
        raise ValueError(name)
    return p + b, p + np.abs(b)


def gated(x, w, bias=None, act="silu"):
    """(h, g, u) from the operands' values; w: gate columns, then up columns."""
    v = x @ w
    if bias is not None:
        v = v + bias
    g, u = np.split(v, 2, axis=1)
    return activation(g, act) * u, g, u


def gated_backward(dh, g, u, act):
    """(dgu, magnitude) before the rounding to bf16."""
    s, smag = activation_slope(g, act)
    a = activation(g, act)
    return np.concatenate([dh * u * s, dh * a], 1), np.concatenate([np.abs(dh * u) * smag, np.abs(dh * a)], 1)


# ---- adapters of many requests -----------------------------------------------------------
def lora(x, a, b, scale, ids, offsets, residual, y):
    """(y, magnitude): y's rows of the sequences are overwritten, the others stay; magnitude: the sum of the
    absolute values of the adapters' terms."""
    T, n = x.shape[0], a.shape[0]
    y, mag = y.copy(), np.zeros_like(y)
    off = np.arange(T + 1) if offsets is None else np.clip(offsets, 0, T)
    for i, lo, hi in zip(ids, off, off[1:]):
        if hi <= lo:
            continue
        y[lo:hi] = 0 if residual is None else residual[lo:hi]
        if 0 <= i < n:
            y[lo:hi] += scale[i] * ((x[lo:hi] @ a[i].T) @ b[i].T)
            mag[lo:hi] = np.abs(scale[i]) * ((np.abs(x[lo:hi]) @ np.abs(a[i]).T) @ np.abs(b[i]).T)
    return y, mag
