"""Thin ctypes binding of the operators around the expert step (include/moe_fp8.h, last part).

Like binding.py: torch tensors on the GPU in, one C call on the current HIP stream, no step of the
computation here and no fallback.  Every operator has a class that holds its argument struct,
output buffers and workspace, so that repeated calls (a layer run every step, graph capture) only
re-issue the C call, and a function of the C entry point's name that builds one and calls it once.
A captured graph and a call beside it that may overlap need an object each: they share nothing then.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as B
from .binding import RouteParams, _check, _need, _ptr, lib, workspace

MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH = range(5)
ACTIVATIONS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU,
               "gelu_tanh": MOE_ACT_GELU_TANH}

_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class AddRmsNormArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("x", _vp), ("ld_x", _i64), ("residual", _vp), ("ld_residual", _i64),
                ("weight", _vp), ("eps", _f32), ("h", _vp), ("y", _vp), ("yq", _vp), ("ys", _vp), ("quant", _i32),
                ("stream", _vp)]


class AddRmsNormBackwardArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("dy", _vp), ("h", _vp), ("weight", _vp), ("eps", _f32), ("dh", _vp),
                ("dx", _vp), ("dweight", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("stream", _vp)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("K", _i32), ("N", _i32), ("xq", _vp), ("xs", _vp), ("w", _vp), ("w_scale", _vp),
                ("bias", _vp), ("activation", _i32), ("residual", _vp), ("ld_residual", _i64), ("y", _vp),
                ("ld_y", _i64), ("out_dtype", _i32), ("quant", _i32), ("workspace", _vp), ("workspace_bytes", _sz),
                ("stream", _vp)]


class BalanceLossArgs(ctypes.Structure):
    _fields_ = [("route", ctypes.POINTER(RouteParams)), ("T", _i32), ("num_seqs", _i32), ("router_logits", _vp),
                ("topk_ids", _vp), ("seq_offsets", _vp), ("balance_coef", _f32), ("z_coef", _f32), ("losses", _vp),
                ("counts", _vp), ("mean_probs", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("stream", _vp)]


class RouteBackwardArgs(ctypes.Structure):
    _fields_ = [("route", ctypes.POINTER(RouteParams)), ("T", _i32), ("num_seqs", _i32), ("router_logits", _vp),
                ("topk_ids", _vp), ("dtopk_weights", _vp), ("counts", _vp), ("seq_offsets", _vp),
                ("balance_coef", _f32), ("z_coef", _f32), ("dlogits", _vp), ("stream", _vp)]


class CombineBackwardArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("k", _i32), ("H", _i32), ("dtype", _i32), ("dy", _vp), ("expert_out", _vp),
                ("assign_pos", _vp), ("topk_weights", _vp), ("dtopk_weights", _vp), ("dexpert_out", _vp),
                ("stream", _vp), ("clear_rows", _i32)]


# The current device and a device's current stream as plain integers, without building a Stream object
# per call (a decode-sized call takes less time on the GPU than that takes on the host).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _Call:
    """An operator's argument struct, its buffers and their device."""

    def _hold(self, fn: str, args: ctypes.Structure, tensors, keep=()) -> None:
        tensors = [t for t in tensors if t is not None]
        dev = tensors[0].device
        for t in tensors:
            if t.device != dev:
                raise ValueError(f"{fn}: all tensors must be on one device, got {dev} and {t.device}")
        self._fn, self.args, self._ref = getattr(lib(), fn), args, ctypes.byref(args)
        self._keep, self._dev = (tensors, keep), dev.index

    def _run(self, stream: Optional[int]) -> None:
        dev = self._dev
        if _current_device() != dev:   # run on the tensors' device, on its own current stream
            with torch.cuda.device(dev):
                return self._run(stream)
        self.args.stream = _raw_stream(dev) if stream is None else stream
        rc = self._fn(self._ref)
        if rc:
            _check(rc)


def _rows(t: torch.Tensor, name: str, dtype, shape) -> int:
    """Checks a matrix whose rows may be strided (last dimension contiguous); its row stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: must be a GPU tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _quant_group(quant: int) -> int:
    return 128 if quant == B.MOE_QUANT_FP8_BLOCK128 else 32


class MoeAddRmsNorm(_Call):
    """h = bf16(x + residual), y = bf16(h * rsqrt(mean(h^2) + eps) * weight) and y's E4M3 codes.

    x, residual: bf16 [T, H], rows may be strided.  weight: float32 [H].
    quant: None for no codes, else the scheme whose activation format yq, ys take
    (MOE_QUANT_FP8_BLOCK128: [T, H/128] scales; MOE_QUANT_MXFP8, MOE_QUANT_W4A8: [T, H/32]).
    want_y: whether y is written.  h: the tensor that receives h (it may be residual or x itself); by
    default a new one where there is a residual, none without.
    A call returns {"h", "y", "yq", "ys"}, None for what is not computed."""

    def __init__(self, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, quant: Optional[int] = None, want_y: bool = True,
                 h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
        T, H = x.shape
        ldx = _rows(x, "x", torch.bfloat16, (T, H))
        ldr = _rows(residual, "residual", torch.bfloat16, (T, H)) if residual is not None else H
        _need(weight, "weight", torch.float32, (H,))
        new = dict(device=x.device)
        if h is None and residual is not None:
            h = torch.empty(T, H, dtype=torch.bfloat16, **new)
        if y is None and want_y:
            y = torch.empty(T, H, dtype=torch.bfloat16, **new)
        for t, name in ((h, "h"), (y, "y")):
            if t is not None:
                _need(t, name, torch.bfloat16, (T, H))
        yq = ys = None
        if quant is not None:
            yq = torch.empty(T, H, dtype=torch.uint8, **new)
            ys = torch.empty(T, max(H // _quant_group(quant), 1), dtype=torch.uint8, **new)
        self.h, self.y, self.yq, self.ys = h, y, yq, ys
        self.out = {"h": h, "y": y, "yq": yq, "ys": ys}
        self._hold("moe_add_rmsnorm",
                   AddRmsNormArgs(T, H, _ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), eps, _ptr(h), _ptr(y), _ptr(yq),
                                  _ptr(ys), quant or 0, None), (x, residual, weight, h, y, yq, ys))

    def __call__(self, stream: Optional[int] = None) -> dict:
        self._run(stream)
        return self.out


def moe_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                    quant: Optional[int] = None, want_y: bool = True, h: Optional[torch.Tensor] = None) -> dict:
    """One call of MoeAddRmsNorm."""
    return MoeAddRmsNorm(x, weight, eps, residual, quant, want_y, h)()


class MoeAddRmsNormBackward(_Call):
    """Gradients of MoeAddRmsNorm from dy (of y) and dh (of h, optional), all bf16 [T, H]; h is what the
    forward call returned (x where it had no residual).  A call returns {"dx", "dweight"}: dx is the
    gradient of x and of the residual; dweight is float32 [H], None with want_dweight=False."""

    def __init__(self, dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 dh: Optional[torch.Tensor] = None, want_dweight: bool = True, dx: Optional[torch.Tensor] = None):
        T, H = h.shape
        for t, name in ((h, "h"), (dy, "dy"), (dh, "dh"), (dx, "dx")):
            if t is not None:
                _need(t, name, torch.bfloat16, (T, H))
        _need(weight, "weight", torch.float32, (H,))
        dx = torch.empty_like(h) if dx is None else dx
        dw = torch.empty(H, dtype=torch.float32, device=h.device) if want_dweight else None
        ws = workspace(lib().moe_add_rmsnorm_backward_workspace_size(T, H), h.device) if want_dweight else None
        self.out = {"dx": dx, "dweight": dw}
        self._hold("moe_add_rmsnorm_backward",
                   AddRmsNormBackwardArgs(T, H, _ptr(dy), _ptr(h), _ptr(weight), eps, _ptr(dh), _ptr(dx), _ptr(dw),
                                          _ptr(ws), ws.numel() if ws is not None else 0, None),
                   (dy, h, weight, dh, dx, dw, ws))

    def __call__(self, stream: Optional[int] = None) -> dict:
        self._run(stream)
        return self.out


def moe_add_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                             dh: Optional[torch.Tensor] = None, want_dweight: bool = True) -> dict:
    """One call of MoeAddRmsNormBackward."""
    return MoeAddRmsNormBackward(dy, h, weight, eps, dh, want_dweight)()


@dataclass
class LinearWeights:
    """Packed weights of one [K, N] product, their scales and an optional float32 bias [N]."""
    K: int
    N: int
    w: torch.Tensor         # packed [K*N]
    w_scale: torch.Tensor   # logical [K/128, ceil(N/128)], or the packed MX scales
    quant: int = B.MOE_QUANT_FP8_BLOCK128
    bias: Optional[torch.Tensor] = None

    @staticmethod
    def from_logical(q: torch.Tensor, scale: torch.Tensor, quant: int = B.MOE_QUANT_FP8_BLOCK128,
                     bias: Optional[torch.Tensor] = None) -> "LinearWeights":
        """E4M3 codes [K, N] with UE8M0 scales [K/128, ceil(N/128)] (MOE_QUANT_FP8_BLOCK128) or
        [K/32, N] (MOE_QUANT_MXFP8)."""
        K, N = q.shape
        if bias is not None:
            _need(bias, "bias", torch.float32, (N,))
        if quant == B.MOE_QUANT_MXFP8:
            _need(scale, "scale", torch.uint8, (K // 32, N))
            w, s = B.moe_prepack_weights_mx(q[None], scale[None], B.MOE_WFMT_E4M3)
        elif quant == B.MOE_QUANT_FP8_BLOCK128:
            _need(scale, "scale", torch.uint8, (K // 128, -(-N // 128)))
            w, s = B.moe_prepack_weights(q[None]), scale
        else:
            raise ValueError("quant must be MOE_QUANT_FP8_BLOCK128 or MOE_QUANT_MXFP8")
        return LinearWeights(K, N, w, s, quant, bias)

    @staticmethod
    def from_float(w: torch.Tensor, quant: int = B.MOE_QUANT_FP8_BLOCK128,
                   bias: Optional[torch.Tensor] = None) -> "LinearWeights":
        """float32 [K, N] -> quantised and packed."""
        N = w.shape[1]
        if quant == B.MOE_QUANT_MXFP8:
            q, s = B.moe_quant_weight_mx(w[None], B.MOE_WFMT_E4M3)
        else:
            if N % 128:   # a block that ends behind column N is quantised as if zeros followed
                w = torch.cat([w, w.new_zeros(w.shape[0], -N % 128)], 1)
            q, s = B.moe_quant_weight_blocks(w[None])
        return LinearWeights.from_logical(q[0][:, :N].contiguous(), s[0], quant, bias)


class MoeLinear(_Call):
    """y = act(dequant(xq, xs) @ w + bias) + residual.

    xq uint8 [T, K] E4M3 and xs uint8 [T, K/128] or [T, K/32] UE8M0 (moe_quant_act / moe_quant_act_mx /
    moe_add_rmsnorm of the weights' scheme); activation one of ACTIVATIONS; residual and y [T, N] of
    out_dtype (bfloat16 or float32), rows may be strided; y may be residual itself."""

    def __init__(self, xq: torch.Tensor, xs: torch.Tensor, w: LinearWeights, activation: str = "none",
                 residual: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, y: Optional[torch.Tensor] = None):
        T = xq.shape[0]
        K, N = w.K, w.N
        _need(xq, "xq", torch.uint8, (T, K))
        _need(xs, "xs", torch.uint8, (T, K // _quant_group(w.quant)))
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation: expected one of {sorted(ACTIVATIONS)}, got {activation!r}")
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype: expected float32 or bfloat16, got {out_dtype}")
        dt = B.MOE_DTYPE_F32 if out_dtype == torch.float32 else B.MOE_DTYPE_BF16
        # (the packed sizes; shapes that the packing refuses are refused by the call)
        sizes = {"w": K * N, "w_scale": K * N // 32 if w.quant == B.MOE_QUANT_MXFP8 else K // 128 * -(-N // 128)}
        for name, n in sizes.items():
            t = getattr(w, name)
            _need(t, name, torch.uint8)
            if t.numel() != n:
                raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")
        if w.bias is not None:
            _need(w.bias, "bias", torch.float32, (N,))
        ldr = _rows(residual, "residual", out_dtype, (T, N)) if residual is not None else N
        if y is None:   # (rows 8 elements apart: N is a multiple of 16)
            y = torch.empty(T, N, dtype=out_dtype, device=xq.device)
        ldy = _rows(y, "y", out_dtype, (T, N))
        nbytes = lib().moe_linear_workspace_size(T, K, N, w.quant)
        ws = workspace(nbytes, xq.device) if nbytes else None
        self.y = y
        self._hold("moe_linear",
                   LinearArgs(T, K, N, _ptr(xq), _ptr(xs), _ptr(w.w), _ptr(w.w_scale), _ptr(w.bias),
                              ACTIVATIONS[activation], _ptr(residual), ldr, _ptr(y), ldy, dt, w.quant, _ptr(ws),
                              ws.numel() if ws is not None else 0, None),
                   (xq, xs, w.w, w.w_scale, w.bias, residual, y, ws))

    def __call__(self, stream: Optional[int] = None) -> torch.Tensor:
        self._run(stream)
        return self.y


def moe_linear(xq: torch.Tensor, xs: torch.Tensor, w: LinearWeights, activation: str = "none",
               residual: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One call of MoeLinear."""
    return MoeLinear(xq, xs, w, activation, residual, out_dtype, y)()


def _router_inputs(params: RouteParams, logits: torch.Tensor, ids: Optional[torch.Tensor],
                   seq_offsets: Optional[torch.Tensor]) -> int:
    T = logits.shape[0]
    _need(logits, "router_logits", torch.float32, (T, params.num_experts))
    if ids is not None:
        _need(ids, "topk_ids", torch.int32, (T, params.top_k))
    if seq_offsets is None:
        return 1
    if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError("seq_offsets: expected shape [num_seqs + 1] with num_seqs >= 1")
    _need(seq_offsets, "seq_offsets", torch.int32)
    return seq_offsets.numel() - 1


class MoeBalanceLoss(_Call):
    """Load-balance and z losses over packed sequences, with counts.

    router_logits float32 [T, E]; topk_ids int32 [T, k] (moe_route); seq_offsets int32
    [num_seqs + 1] on the GPU, or None for one sequence of all rows.  A call returns {"losses":
    float32 [3] (sum, balance, z), "counts": int32 [num_seqs, E], "mean_probs": float32 [num_seqs, E]}."""

    def __init__(self, params: RouteParams, router_logits: torch.Tensor, topk_ids: torch.Tensor,
                 seq_offsets: Optional[torch.Tensor] = None, balance_coef: float = 1e-2, z_coef: float = 0.0):
        params = RouteParams.from_buffer_copy(params)   # as they were when the buffers were checked against them
        S = _router_inputs(params, router_logits, topk_ids, seq_offsets)
        T, E, dev = router_logits.shape[0], params.num_experts, router_logits.device
        self.losses = torch.empty(3, dtype=torch.float32, device=dev)
        self.counts = torch.empty(S, E, dtype=torch.int32, device=dev)
        self.mean_probs = torch.empty(S, E, dtype=torch.float32, device=dev)
        ws = workspace(lib().moe_balance_loss_workspace_size(T, E, S), dev)
        self.out = {"losses": self.losses, "counts": self.counts, "mean_probs": self.mean_probs}
        self._hold("moe_balance_loss",
                   BalanceLossArgs(ctypes.pointer(params), T, S, _ptr(router_logits), _ptr(topk_ids), _ptr(seq_offsets),
                                   balance_coef, z_coef, _ptr(self.losses), _ptr(self.counts), _ptr(self.mean_probs),
                                   _ptr(ws), ws.numel(), None),
                   (router_logits, topk_ids, seq_offsets, self.losses, self.counts, self.mean_probs, ws), params)

    def __call__(self, stream: Optional[int] = None) -> dict:
        self._run(stream)
        return self.out


def moe_balance_loss(params: RouteParams, router_logits: torch.Tensor, topk_ids: torch.Tensor,
                     seq_offsets: Optional[torch.Tensor] = None, balance_coef: float = 1e-2,
                     z_coef: float = 0.0) -> dict:
    """One call of MoeBalanceLoss."""
    return MoeBalanceLoss(params, router_logits, topk_ids, seq_offsets, balance_coef, z_coef)()


class MoeRouteBackward(_Call):
    """The router logits' gradient, float32 [T, E]: through the routing weights from dweights float32
    [T, k] (None: not), and through the losses of moe_balance_loss from its counts (None: the z loss
    alone), with the same seq_offsets and coefficients."""

    def __init__(self, params: RouteParams, router_logits: torch.Tensor, topk_ids: Optional[torch.Tensor] = None,
                 dweights: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                 seq_offsets: Optional[torch.Tensor] = None, balance_coef: float = 1e-2, z_coef: float = 0.0,
                 dlogits: Optional[torch.Tensor] = None):
        params = RouteParams.from_buffer_copy(params)   # as they were when the buffers were checked against them
        S = _router_inputs(params, router_logits, topk_ids, seq_offsets)
        T, E = router_logits.shape
        if dweights is not None:
            if topk_ids is None:
                raise ValueError("dweights needs topk_ids")
            _need(dweights, "dweights", torch.float32, (T, params.top_k))
        if counts is not None:
            _need(counts, "counts", torch.int32, (S, E))
        if dlogits is None:
            dlogits = torch.empty_like(router_logits)
        _need(dlogits, "dlogits", torch.float32, (T, E))
        self.dlogits = dlogits
        self._hold("moe_route_backward",
                   RouteBackwardArgs(ctypes.pointer(params), T, S, _ptr(router_logits), _ptr(topk_ids), _ptr(dweights),
                                     _ptr(counts), _ptr(seq_offsets), balance_coef, z_coef, _ptr(dlogits), None),
                   (router_logits, topk_ids, dweights, counts, seq_offsets, dlogits), params)

    def __call__(self, stream: Optional[int] = None) -> torch.Tensor:
        self._run(stream)
        return self.dlogits


def moe_route_backward(params: RouteParams, router_logits: torch.Tensor, topk_ids: Optional[torch.Tensor] = None,
                       dweights: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                       seq_offsets: Optional[torch.Tensor] = None, balance_coef: float = 1e-2,
                       z_coef: float = 0.0) -> torch.Tensor:
    """One call of MoeRouteBackward."""
    return MoeRouteBackward(params, router_logits, topk_ids, dweights, counts, seq_offsets, balance_coef, z_coef)()


class MoeCombineBackward(_Call):
    """Gradients of moe_combine from dy bf16 [T, H].  A call returns {"dweights": float32 [T, k] (None
    with want_dweights=False), "d_expert_out": [T*k, H] of expert_out's dtype (None unless asked for)}.

    d_expert_out: False, True (a new tensor) or the tensor to write (it may be expert_out itself).  Every
    call sets the rows of a new tensor that assign_pos does not name to 0; those of a given one are left
    as they are."""

    def __init__(self, dy: torch.Tensor, expert_out: torch.Tensor, assign_pos: torch.Tensor, topk_weights: torch.Tensor,
                 d_expert_out=False, want_dweights: bool = True):
        T, k = topk_weights.shape
        H = dy.shape[1]
        _need(dy, "dy", torch.bfloat16, (T, H))
        if expert_out.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"expert_out: expected float32 or bfloat16, got {expert_out.dtype}")
        _need(expert_out, "expert_out", expert_out.dtype, (T * k, H))
        _need(topk_weights, "topk_weights", torch.float32, (T, k))
        if assign_pos.numel() != T * k:
            raise ValueError(f"assign_pos: expected {T * k} entries, got {assign_pos.numel()}")
        _need(assign_pos, "assign_pos", torch.int32)
        deo = None
        if isinstance(d_expert_out, torch.Tensor):
            deo = d_expert_out
            _need(deo, "d_expert_out", expert_out.dtype, (T * k, H))
        elif d_expert_out:
            deo = torch.empty_like(expert_out)
        dw = torch.empty(T, k, dtype=torch.float32, device=dy.device) if want_dweights else None
        dt = B.MOE_DTYPE_BF16 if expert_out.dtype == torch.bfloat16 else B.MOE_DTYPE_F32
        self.out = {"dweights": dw, "d_expert_out": deo}
        self._hold("moe_combine_backward",
                   CombineBackwardArgs(T, k, H, dt, _ptr(dy), _ptr(expert_out), _ptr(assign_pos), _ptr(topk_weights),
                                       _ptr(dw), _ptr(deo), None, int(deo is not None and deo is not d_expert_out)),
                   (dy, expert_out, assign_pos, topk_weights, dw, deo))

    def __call__(self, stream: Optional[int] = None) -> dict:
        self._run(stream)
        return self.out


def moe_combine_backward(dy: torch.Tensor, expert_out: torch.Tensor, assign_pos: torch.Tensor,
                         topk_weights: torch.Tensor, d_expert_out=False, want_dweights: bool = True) -> dict:
    """One call of MoeCombineBackward."""
    return MoeCombineBackward(dy, expert_out, assign_pos, topk_weights, d_expert_out, want_dweights)()
