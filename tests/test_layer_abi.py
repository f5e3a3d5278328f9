"""Refusals of the operators around the expert step, without a GPU: every bad argument is turned
down on the host before any HIP call, with the code and text that name it."""
import ctypes

import pytest

import mixture_experts_fp8_amd as M
from mixture_experts_fp8_amd import binding as B
from mixture_experts_fp8_amd import layer as L

A = 0x10000000          # never dereferenced; buffers far apart
BIG = 1 << 33


def at(i, off=0):
    return A + i * BIG + off


def call(name, struct, defaults, **over):
    a = dict(defaults)
    a.update(over)
    return getattr(M.lib(), name)(ctypes.byref(struct(**a)))


NORM = dict(T=4, H=256, x=at(0), ld_x=256, residual=at(1), ld_residual=256, weight=at(2), eps=1e-6, h=at(3), y=at(4),
            yq=at(5), ys=at(6), quant=0)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=0), B.MOE_ERR_INVALID, "T (0)"), (dict(H=0), B.MOE_ERR_INVALID, "H (0)"),
    (dict(H=252, ld_x=256), B.MOE_ERR_UNSUPPORTED, "multiple of 8"),
    (dict(H=65536, ld_x=65536, ld_residual=65536), B.MOE_ERR_UNSUPPORTED, "32768"),
    (dict(eps=-1.0), B.MOE_ERR_INVALID, "eps"), (dict(eps=float("nan")), B.MOE_ERR_INVALID, "eps"),
    (dict(x=None), B.MOE_ERR_INVALID, "x and weight"), (dict(weight=None), B.MOE_ERR_INVALID, "x and weight"),
    (dict(h=None, y=None, yq=None, ys=None), B.MOE_ERR_INVALID, "must be given"),
    (dict(ys=None), B.MOE_ERR_INVALID, "together"), (dict(yq=None), B.MOE_ERR_INVALID, "together"),
    (dict(quant=3), B.MOE_ERR_INVALID, "quantises activations"), (dict(quant=-1), B.MOE_ERR_INVALID, "quant"),
    (dict(H=200), B.MOE_ERR_UNSUPPORTED, "multiple of 128"), (dict(H=200, quant=1), B.MOE_ERR_UNSUPPORTED, "multiple of 32"),
    (dict(ld_x=128), B.MOE_ERR_INVALID, "ld_x"), (dict(ld_residual=0), B.MOE_ERR_INVALID, "ld_residual"),
    (dict(ld_x=260), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(x=at(0, 8)), B.MOE_ERR_UNSUPPORTED, "aligned"),
    (dict(weight=at(2, 4)), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(y=at(4, 2)), B.MOE_ERR_UNSUPPORTED, "aligned"),
    (dict(yq=at(5, 4)), B.MOE_ERR_UNSUPPORTED, "8-byte"),
    (dict(h=at(0, 512)), B.MOE_ERR_INVALID, "overlap"), (dict(h=at(0), ld_x=264), B.MOE_ERR_INVALID, "overlap"),
    (dict(y=at(1)), B.MOE_ERR_INVALID, "overlap"), (dict(y=at(3)), B.MOE_ERR_INVALID, "h and y"),
    (dict(h=at(0), y=at(0)), B.MOE_ERR_INVALID, "h and y"), (dict(yq=at(2)), B.MOE_ERR_INVALID, "weight"),
    (dict(ys=at(5, 1016)), B.MOE_ERR_INVALID, "yq and ys"),
])
def test_add_rmsnorm_refuses(over, code, needle):
    assert call("moe_add_rmsnorm", L.AddRmsNormArgs, NORM, **over) == code
    assert needle in M.moe_last_error() and "moe_add_rmsnorm" in M.moe_last_error()


NBWD = dict(T=4, H=256, dy=at(0), h=at(1), weight=at(2), eps=1e-6, dh=at(3), dx=at(4), dweight=at(5), workspace=at(6),
            workspace_bytes=1 << 20)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=-1), B.MOE_ERR_INVALID, "T (-1)"), (dict(H=12), B.MOE_ERR_UNSUPPORTED, "multiple of 8"),
    (dict(dx=None), B.MOE_ERR_INVALID, "dx"), (dict(dh=at(3, 8)), B.MOE_ERR_UNSUPPORTED, "aligned"),
    (dict(dweight=at(5, 2)), B.MOE_ERR_INVALID, "dweight"), (dict(workspace=None), B.MOE_ERR_WORKSPACE, "workspace"),
    (dict(workspace_bytes=1023), B.MOE_ERR_WORKSPACE, "need 1024"), (dict(workspace=at(6, 64)), B.MOE_ERR_INVALID, "256-byte"),
    (dict(dx=at(1)), B.MOE_ERR_INVALID, "dx must not overlap h"), (dict(dx=at(0, 512)), B.MOE_ERR_INVALID, "dx must not overlap dy"),
    (dict(dweight=at(2)), B.MOE_ERR_INVALID, "dweight must not overlap weight"),
    (dict(workspace=at(4)), B.MOE_ERR_INVALID, "dx and workspace"),
])
def test_add_rmsnorm_backward_refuses(over, code, needle):
    assert call("moe_add_rmsnorm_backward", L.AddRmsNormBackwardArgs, NBWD, **over) == code
    assert needle in M.moe_last_error()


LIN = dict(T=4, K=256, N=144, xq=at(0), xs=at(1), w=at(2), w_scale=at(3), bias=at(4), activation=0, residual=at(5),
           ld_residual=144, y=at(6), ld_y=144, out_dtype=1, quant=0, workspace=at(7), workspace_bytes=1 << 30)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=0), B.MOE_ERR_INVALID, "T, K, N"), (dict(K=200), B.MOE_ERR_UNSUPPORTED, "multiple of 128"),
    (dict(K=65536), B.MOE_ERR_UNSUPPORTED, "32768"), (dict(N=24), B.MOE_ERR_UNSUPPORTED, "multiple of 16"),
    (dict(T=1 << 23), B.MOE_ERR_UNSUPPORTED, "2^31"), (dict(N=1 << 23, ld_y=1 << 23, ld_residual=1 << 23), B.MOE_ERR_UNSUPPORTED, "2^31"),
    (dict(quant=2), B.MOE_ERR_UNSUPPORTED, "quant"), (dict(quant=3), B.MOE_ERR_UNSUPPORTED, "quant"),
    (dict(quant=7), B.MOE_ERR_INVALID, "quant"), (dict(activation=5), B.MOE_ERR_INVALID, "activation"),
    (dict(out_dtype=2), B.MOE_ERR_INVALID, "out_dtype"), (dict(w_scale=None), B.MOE_ERR_INVALID, "w_scale"),
    (dict(ld_y=128), B.MOE_ERR_INVALID, "ld_y"), (dict(ld_residual=128), B.MOE_ERR_INVALID, "ld_residual"),
    (dict(ld_y=148), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(y=at(6, 8)), B.MOE_ERR_UNSUPPORTED, "aligned"),
    (dict(xq=at(0, 8)), B.MOE_ERR_UNSUPPORTED, "xq and w"), (dict(quant=1, xs=at(1, 2)), B.MOE_ERR_UNSUPPORTED, "xs and w_scale"),
    (dict(bias=at(4, 2)), B.MOE_ERR_INVALID, "bias"), (dict(y=at(5), ld_y=160), B.MOE_ERR_INVALID, "overlap"),
    (dict(y=at(5, 16)), B.MOE_ERR_INVALID, "overlap"), (dict(y=at(0)), B.MOE_ERR_INVALID, "xq"),
])
def test_linear_refuses(over, code, needle):
    assert call("moe_linear", L.LinearArgs, LIN, **over) == code
    assert needle in M.moe_last_error()


def _route(**kw):
    p = M.route_params(**{**dict(num_experts=8, top_k=2), **kw})
    _route.keep = p
    return ctypes.pointer(p)


BAL = dict(T=16, num_seqs=2, router_logits=at(0), topk_ids=at(1), seq_offsets=at(2), balance_coef=0.1, z_coef=0.1,
           losses=at(3), counts=at(4), mean_probs=at(5), workspace=at(6), workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,over,code,needle", [
    ({}, dict(T=0), B.MOE_ERR_INVALID, "T (0)"), (dict(top_k=9), {}, B.MOE_ERR_INVALID, "top_k"),
    (dict(num_experts=2000), {}, B.MOE_ERR_UNSUPPORTED, "exceeds max"), ({}, dict(num_seqs=0), B.MOE_ERR_INVALID, "num_seqs"),
    ({}, dict(seq_offsets=None), B.MOE_ERR_INVALID, "without seq_offsets"), ({}, dict(num_seqs=1 << 21), B.MOE_ERR_UNSUPPORTED, "num_seqs"),
    ({}, dict(router_logits=None), B.MOE_ERR_INVALID, "router_logits"), ({}, dict(topk_ids=None), B.MOE_ERR_INVALID, "topk_ids"),
    ({}, dict(balance_coef=float("inf")), B.MOE_ERR_INVALID, "finite"), ({}, dict(z_coef=float("nan")), B.MOE_ERR_INVALID, "finite"),
    ({}, dict(workspace_bytes=8), B.MOE_ERR_WORKSPACE, "need"), ({}, dict(workspace=at(6, 16)), B.MOE_ERR_INVALID, "256-byte"),
    ({}, dict(counts=at(1)), B.MOE_ERR_INVALID, "overlap"), ({}, dict(mean_probs=at(4)), B.MOE_ERR_INVALID, "counts and mean_probs"),
    (dict(top_k=8), dict(T=1 << 27), B.MOE_ERR_UNSUPPORTED, "2^29"), ({}, dict(router_logits=at(0, 2)), B.MOE_ERR_INVALID, "aligned"),
])
def test_balance_loss_refuses(kw, over, code, needle):
    assert call("moe_balance_loss", L.BalanceLossArgs, dict(BAL, route=_route(**kw)), **over) == code
    assert needle in M.moe_last_error()


RB = dict(T=16, num_seqs=1, router_logits=at(0), topk_ids=at(1), dtopk_weights=at(2), counts=at(3), seq_offsets=None,
          balance_coef=0.1, z_coef=0.1, dlogits=at(5))


@pytest.mark.parametrize("kw,over,code,needle", [
    ({}, dict(dlogits=None), B.MOE_ERR_INVALID, "dlogits"), ({}, dict(topk_ids=None), B.MOE_ERR_INVALID, "needs topk_ids"),
    ({}, dict(num_seqs=3), B.MOE_ERR_INVALID, "num_seqs"), (dict(routed_scaling_factor=float("inf")), {}, B.MOE_ERR_INVALID, "finite"),
    ({}, dict(dlogits=at(0, 16)), B.MOE_ERR_INVALID, "overlap"), ({}, dict(dlogits=at(2)), B.MOE_ERR_INVALID, "dtopk_weights"),
])
def test_route_backward_refuses(kw, over, code, needle):
    assert call("moe_route_backward", L.RouteBackwardArgs, dict(RB, route=_route(**kw)), **over) == code
    assert needle in M.moe_last_error()


CB = dict(T=4, k=2, H=256, dtype=1, dy=at(0), expert_out=at(1), assign_pos=at(2), topk_weights=at(3), dtopk_weights=at(4),
          dexpert_out=at(5))


@pytest.mark.parametrize("over,code,needle", [
    (dict(k=0), B.MOE_ERR_INVALID, "T, k, H"), (dict(H=100), B.MOE_ERR_UNSUPPORTED, "multiple of 8"),
    (dict(dtype=4), B.MOE_ERR_INVALID, "dtype"), (dict(T=1 << 28), B.MOE_ERR_UNSUPPORTED, "2^29"),
    (dict(dy=None), B.MOE_ERR_INVALID, "dy"), (dict(dtopk_weights=None, dexpert_out=None), B.MOE_ERR_INVALID, "must be given"),
    (dict(expert_out=None), B.MOE_ERR_INVALID, "needs expert_out"), (dict(topk_weights=None), B.MOE_ERR_INVALID, "needs topk_weights"),
    (dict(dexpert_out=at(5, 8)), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(dexpert_out=at(0)), B.MOE_ERR_INVALID, "overlap"),
    (dict(dexpert_out=at(1, 16)), B.MOE_ERR_INVALID, "expert_out"), (dict(dtopk_weights=at(3)), B.MOE_ERR_INVALID, "topk_weights"),
])
def test_combine_backward_refuses(over, code, needle):
    assert call("moe_combine_backward", L.CombineBackwardArgs, CB, **over) == code
    assert needle in M.moe_last_error()


@pytest.mark.parametrize("name", ["moe_add_rmsnorm", "moe_add_rmsnorm_backward", "moe_linear", "moe_balance_loss",
                                  "moe_route_backward", "moe_combine_backward"])
def test_null_args(name):
    assert getattr(M.lib(), name)(None) == B.MOE_ERR_INVALID and "args" in M.moe_last_error()


def test_workspace_sizes():
    L_ = M.lib()
    assert L_.moe_add_rmsnorm_backward_workspace_size(5, 256) == 2 * 256 * 4   # four rows per workgroup
    assert L_.moe_add_rmsnorm_backward_workspace_size(5, 2048) == 5 * 2048 * 4
    assert L_.moe_add_rmsnorm_backward_workspace_size(0, 256) == 0
    assert L_.moe_balance_loss_workspace_size(0, 8, 1) == 0
    small, large = (L_.moe_balance_loss_workspace_size(T, 128, 3) for T in (64, 16384))
    assert 0 < small < large
