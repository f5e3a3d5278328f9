"""The operators around the expert step (CPU, float64): residual + RMS norm, FP8 linear, router
losses and the gradients of the norm, the router logits and the combine.

TEST INFRASTRUCTURE ONLY: nothing in the product path may import this module.

Definitions as stated in include/moe_fp8.h.  Pins (tests/test_oracle_layer.py): the gradients agree
with central differences of the forward functions here; closed forms (a uniform router has balance
loss equal to its coefficient; a one-hot weight picks an input column); hand values.
"""
from __future__ import annotations

import math

import numpy as np

from . import codec, mx
from .w8a16 import bf16_rne

_erf = np.vectorize(math.erf, otypes=[np.float64])


# ---- residual + RMS norm -----------------------------------------------------------------
def add_rmsnorm(x, residual, weight, eps):
    """(h, y) float64: h rounded to bf16, y not rounded."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = bf16_rne(h + residual)
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h, h * r * weight


def rmsnorm_backward(dy, h, weight, eps, dh=None):
    """(dx, dweight, dx_mag, dw_mag): the gradients and the sums of the absolute values of the terms
    that they are made of."""
    H = h.shape[1]
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    xh, g = h * r, dy * weight
    dx = r * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    mag = r * (np.abs(g) + np.abs(xh) * np.abs(g * xh).sum(axis=1, keepdims=True) / H)
    if dh is not None:
        dx, mag = dx + dh, mag + np.abs(dh)
    return dx, (dy * xh).sum(axis=0), mag, np.abs(dy * xh).sum(axis=0)


# ---- linear ------------------------------------------------------------------------------
def activation(v, name):
    v = np.asarray(v, dtype=np.float64)
    if name == "none":
        return v
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    raise ValueError(name)


def dequant_linear(xq, xs, wq, ws, micro):
    """Values of the operands: micro = False, scales per (row, 128) and 128 x 128 block (the last
    column block may be short); True, per (row, 32) and (32, column)."""
    K, N = wq.shape
    gs = 32 if micro else 128
    x = codec.e4m3_decode(xq) * np.repeat(codec.ue8m0_decode(xs), gs, axis=1)
    s = np.repeat(codec.ue8m0_decode(ws), gs, axis=0)
    if not micro:
        s = np.repeat(s, 128, axis=1)[:, :N]
    return x, codec.e4m3_decode(wq) * s


def linear(x, w, bias=None, act="none", residual=None):
    """(y, sum of |x| |w|) from the operands' values."""
    v = x @ w
    if bias is not None:
        v = v + bias
    y = activation(v, act)
    return (y if residual is None else y + residual), np.abs(x) @ np.abs(w)


# ---- router losses -----------------------------------------------------------------------
def _scores(logits, scoring):
    """(p [T, E], raw scores, d raw / d logit as a factor of raw): rows without a live logit give 0."""
    l = np.asarray(logits, dtype=np.float64)
    m = l.max(axis=1, keepdims=True)
    num = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    tot = num.sum(axis=1, keepdims=True)
    soft = np.divide(num, tot, out=np.zeros_like(num), where=tot != 0)
    with np.errstate(divide="ignore"):
        lse = np.where(tot[:, 0] != 0, np.where(np.isneginf(m), 0.0, m)[:, 0] + np.log(tot[:, 0]), 0.0)
    if scoring == "softmax":
        return soft, soft, np.ones_like(soft), soft, lse
    with np.errstate(over="ignore"):
        e = np.exp(-l)
    s = 1.0 / (1.0 + e)
    z = s.sum(axis=1, keepdims=True)
    p = np.divide(s, z, out=np.zeros_like(s), where=z != 0)
    return p, s, np.where(np.isinf(e), 1.0, np.where(np.isinf(e), 0.0, e) * s), soft, lse


def _spans(T, offsets):
    off = [0, T] if offsets is None else [min(max(int(o), 0), T) for o in offsets]
    return list(zip(off, off[1:]))


def balance_loss(logits, ids, k, scoring, balance_coef, z_coef, offsets=None):
    """(losses [3], counts [S, E], mean_probs [S, E])."""
    T, E = logits.shape
    spans = _spans(T, offsets)
    counts = np.zeros((len(spans), E), dtype=np.int64)
    mean = np.zeros((len(spans), E))
    bal = z = 0.0
    live = sum(b > a for a, b in spans)
    valid = sum(b - a for a, b in spans)
    for s, (a, b) in enumerate(spans):
        if b <= a:
            continue
        p, _, _, _, lse = _scores(logits[a:b], scoring)
        got = ids[a:b].reshape(-1)
        counts[s] = np.bincount(got[(got >= 0) & (got < E)], minlength=E)
        mean[s] = p.mean(axis=0)
        bal += balance_coef / live * (E / (k * (b - a)) * counts[s] * mean[s]).sum()
        z += z_coef / valid * (lse ** 2).sum()
    return np.array([bal + z, bal, z]), counts, mean


def route_weights(logits, ids, scoring, renorm, rsf):
    """moe_route's weights for given ids [T, k]; dropped ids (outside [0, E)) weigh nothing."""
    T, E = logits.shape
    _, raw, _, _, _ = _scores(logits, scoring)
    ok = (ids >= 0) & (ids < E)
    w = np.where(ok, np.take_along_axis(raw, np.clip(ids, 0, E - 1), axis=1), 0.0)
    if scoring == "sigmoid" or renorm:
        tot = w.sum(axis=1, keepdims=True)
        w = np.divide(w, tot, out=np.zeros_like(w), where=tot != 0)
    return w * rsf


def route_backward(logits, ids, k, scoring, renorm, rsf, dweights=None, counts=None, balance_coef=0.0, z_coef=0.0,
                   offsets=None):
    """(dlogits, sum of the absolute values of its terms)."""
    T, E = logits.shape
    spans = _spans(T, offsets)
    live, valid = sum(b > a for a, b in spans), sum(b - a for a, b in spans)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for s, (a, b) in enumerate(spans):
        if b <= a:
            continue
        p, raw, om, soft, lse = _scores(logits[a:b], scoring)
        n = b - a
        if counts is not None:
            u = balance_coef / live * E / (k * n) * counts[s] / n
            pu = (p * u).sum(axis=1, keepdims=True)
            d[a:b] += p * om * (u - pu)
            mag[a:b] += p * om * (np.abs(u) + np.abs(pu))
        zt = 2.0 * z_coef / valid * lse[:, None] * soft
        d[a:b] += zt
        mag[a:b] += np.abs(zt)
        if dweights is not None:
            D, m, D_abs = np.zeros((n, E)), np.zeros((n, E)), np.zeros((n, E))
            for j in range(k):
                e = ids[a:b, j]
                ok = np.nonzero((e >= 0) & (e < E))[0]
                D[ok, e[ok]] += dweights[a:b][ok, j]
                D_abs[ok, e[ok]] += np.abs(dweights[a:b][ok, j])
                m[ok, e[ok]] += 1
            if scoring == "softmax" and not renorm:
                d[a:b] += rsf * raw * (D - (raw * D).sum(axis=1, keepdims=True))
                mag[a:b] += abs(rsf) * raw * (D_abs + (raw * D_abs).sum(axis=1, keepdims=True))
            else:
                got = np.where(m > 0, raw, 0.0)
                if scoring == "softmax":   # a softmax over the chosen: theirs may all be 0 beside a far larger logit
                    sel = np.where(m > 0, np.asarray(logits[a:b], dtype=np.float64), -np.inf)
                    top = sel.max(axis=1, keepdims=True)
                    got = np.exp(sel - np.where(np.isneginf(top), 0.0, top))
                tot = (m * got).sum(axis=1, keepdims=True)
                q = np.divide(got, tot, out=np.zeros_like(got), where=tot != 0)
                d[a:b] += rsf * q * om * (D - m * (q * D).sum(axis=1, keepdims=True))
                mag[a:b] += abs(rsf) * q * om * (D_abs + m * (q * D_abs).sum(axis=1, keepdims=True))
    return d, mag


# ---- combine -----------------------------------------------------------------------------
def combine_backward(dy, expert_out, pos, weights):
    """(dweights [T, k], sums of absolute products, {row: w dy} for the rows that pos names)."""
    T, k = weights.shape
    pos = pos.reshape(T, k)
    dw, mag, rows = np.zeros((T, k)), np.zeros((T, k)), {}
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < T * k:
                dw[t, j] = dy[t] @ expert_out[pos[t, j]]
                mag[t, j] = np.abs(dy[t]) @ np.abs(expert_out[pos[t, j]])
                rows[int(pos[t, j])] = weights[t, j] * dy[t]
    return dw, mag, rows
