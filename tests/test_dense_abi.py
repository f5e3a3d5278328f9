"""Refusals of the operators of dense layers, without a GPU: every bad argument is turned down on the
host before any HIP call, with the code and text that name it."""
import pytest

import mixture_experts_fp8_amd as M
from mixture_experts_fp8_amd import binding as B
from mixture_experts_fp8_amd import layer as L
from test_layer_abi import at, call

NORM = dict(T=4, H=256, x=at(0), ld_x=256, residual=at(1), ld_residual=256, weight=at(2), bias=at(7), eps=1e-5,
            h=at(3), y=at(4), yq=at(5), ys=at(6), quant=0)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=0), B.MOE_ERR_INVALID, "T (0)"), (dict(H=252, ld_x=256), B.MOE_ERR_UNSUPPORTED, "multiple of 8"),
    (dict(H=65536, ld_x=65536, ld_residual=65536), B.MOE_ERR_UNSUPPORTED, "32768"),
    (dict(eps=float("inf")), B.MOE_ERR_INVALID, "eps"), (dict(weight=None), B.MOE_ERR_INVALID, "x and weight"),
    (dict(h=None, y=None, yq=None, ys=None), B.MOE_ERR_INVALID, "must be given"),
    (dict(ys=None), B.MOE_ERR_INVALID, "together"), (dict(quant=3), B.MOE_ERR_INVALID, "quantises activations"),
    (dict(H=200), B.MOE_ERR_UNSUPPORTED, "multiple of 128"), (dict(ld_x=128), B.MOE_ERR_INVALID, "ld_x"),
    (dict(x=at(0, 8)), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(bias=at(7, 4)), B.MOE_ERR_UNSUPPORTED, "bias"),
    (dict(y=at(7)), B.MOE_ERR_INVALID, "y must not overlap bias"), (dict(h=at(7, 512)), B.MOE_ERR_INVALID, "bias"),
    (dict(y=at(1)), B.MOE_ERR_INVALID, "overlap"), (dict(y=at(3)), B.MOE_ERR_INVALID, "h and y"),
])
def test_add_layernorm_refuses(over, code, needle):
    assert call("moe_add_layernorm", L.AddLayerNormArgs, NORM, **over) == code
    assert needle in M.moe_last_error() and "moe_add_layernorm" in M.moe_last_error()


NBWD = dict(T=4, H=256, dy=at(0), h=at(1), weight=at(2), eps=1e-5, dh=at(3), dx=at(4), dweight=at(5), dbias=at(7),
            workspace=at(6), workspace_bytes=1 << 20)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=-1), B.MOE_ERR_INVALID, "T (-1)"), (dict(H=12), B.MOE_ERR_UNSUPPORTED, "multiple of 8"),
    (dict(dx=None), B.MOE_ERR_INVALID, "dx"), (dict(dbias=at(7, 2)), B.MOE_ERR_INVALID, "dbias"),
    (dict(workspace=None), B.MOE_ERR_WORKSPACE, "workspace"), (dict(workspace=None, dweight=None), B.MOE_ERR_WORKSPACE, "workspace"),
    (dict(workspace_bytes=2047), B.MOE_ERR_WORKSPACE, "need 2048"), (dict(workspace=at(6, 64)), B.MOE_ERR_INVALID, "256-byte"),
    (dict(dx=at(1)), B.MOE_ERR_INVALID, "dx must not overlap h"), (dict(dbias=at(5, 512)), B.MOE_ERR_INVALID, "dweight and dbias"),
    (dict(dbias=at(2)), B.MOE_ERR_INVALID, "dbias must not overlap weight"), (dict(workspace=at(7)), B.MOE_ERR_INVALID, "dbias and workspace"),
])
def test_add_layernorm_backward_refuses(over, code, needle):
    assert call("moe_add_layernorm_backward", L.AddLayerNormBackwardArgs, NBWD, **over) == code
    assert needle in M.moe_last_error() and "moe_add_layernorm_backward" in M.moe_last_error()


@pytest.mark.parametrize("name", ["moe_add_layernorm", "moe_add_layernorm_backward", "moe_gated_linear",
                                  "moe_gated_linear_backward", "moe_lora"])
def test_null_arguments(name):
    assert getattr(M.lib(), name)(None) == B.MOE_ERR_INVALID
    assert name in M.moe_last_error()


GATED = dict(T=4, K=256, I=96, xq=at(0), xs=at(1), w=at(2), w_scale=at(3), bias=at(4), activation=2, h=at(5), gu=at(6), quant=0)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=0), B.MOE_ERR_INVALID, "T, K, I"), (dict(K=200), B.MOE_ERR_UNSUPPORTED, "multiple of 128"),
    (dict(I=48), B.MOE_ERR_UNSUPPORTED, "multiple of 32"), (dict(K=65536), B.MOE_ERR_UNSUPPORTED, "32768"),
    (dict(T=1 << 23), B.MOE_ERR_UNSUPPORTED, "2^31"), (dict(I=1 << 22), B.MOE_ERR_UNSUPPORTED, "2^31"),
    (dict(quant=2), B.MOE_ERR_UNSUPPORTED, "quant"), (dict(quant=9), B.MOE_ERR_INVALID, "quant"),
    (dict(activation=5), B.MOE_ERR_INVALID, "activation"), (dict(activation=-1), B.MOE_ERR_INVALID, "activation"),
    (dict(h=None), B.MOE_ERR_INVALID, "h must not"), (dict(w=None), B.MOE_ERR_INVALID, "w_scale"),
    (dict(h=at(5, 8)), B.MOE_ERR_UNSUPPORTED, "16-byte"), (dict(gu=at(6, 8)), B.MOE_ERR_UNSUPPORTED, "16-byte"),
    (dict(quant=1, xs=at(1, 2)), B.MOE_ERR_UNSUPPORTED, "4-byte"), (dict(bias=at(4, 1)), B.MOE_ERR_INVALID, "bias"),
    (dict(gu=at(5, 256)), B.MOE_ERR_INVALID, "h and gu"), (dict(h=at(0)), B.MOE_ERR_INVALID, "h must not overlap xq"),
    (dict(gu=at(4)), B.MOE_ERR_INVALID, "gu must not overlap bias"),
])
def test_gated_linear_refuses(over, code, needle):
    assert call("moe_gated_linear", L.GatedLinearArgs, GATED, **over) == code
    assert needle in M.moe_last_error() and "moe_gated_linear" in M.moe_last_error()


GBWD = dict(T=4, K=256, I=96, dh=at(0), gu=at(1), activation=2, xq=at(2), xs=at(3), w=at(4), w_scale=at(5), quant=0, dgu=at(6),
            dx=at(7), dw=at(8), dw_dtype=0, dbias=at(9), workspace=at(10), workspace_bytes=1 << 30)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=0), B.MOE_ERR_INVALID, "T, K, I"), (dict(K=200), B.MOE_ERR_UNSUPPORTED, "multiple of 128"),
    (dict(I=48), B.MOE_ERR_UNSUPPORTED, "multiple of 32"), (dict(T=1 << 22), B.MOE_ERR_UNSUPPORTED, "2^30"),
    (dict(quant=3), B.MOE_ERR_UNSUPPORTED, "quant"), (dict(activation=7), B.MOE_ERR_INVALID, "activation"),
    (dict(dgu=None), B.MOE_ERR_INVALID, "dgu"), (dict(gu=None), B.MOE_ERR_INVALID, "gu"),
    (dict(w=None), B.MOE_ERR_INVALID, "dx needs"), (dict(xs=None), B.MOE_ERR_INVALID, "dw needs"),
    (dict(dw_dtype=2), B.MOE_ERR_INVALID, "dw_dtype"), (dict(dx=at(7, 8)), B.MOE_ERR_UNSUPPORTED, "16-byte"),
    (dict(dbias=at(9, 2)), B.MOE_ERR_INVALID, "dbias"), (dict(workspace=None), B.MOE_ERR_WORKSPACE, "workspace"),
    (dict(workspace_bytes=1000), B.MOE_ERR_WORKSPACE, "need"), (dict(workspace=at(10, 128)), B.MOE_ERR_INVALID, "256-byte"),
    (dict(dgu=at(0)), B.MOE_ERR_INVALID, "dgu must not overlap dh"), (dict(dgu=at(1, 256)), B.MOE_ERR_INVALID, "dgu must not overlap gu"),
    (dict(dx=at(1)), B.MOE_ERR_INVALID, "dx must not overlap gu"), (dict(dw=at(7)), B.MOE_ERR_INVALID, "dx and dw"),
    (dict(dw=at(4)), B.MOE_ERR_INVALID, "dw must not overlap w"), (dict(workspace=at(2)), B.MOE_ERR_INVALID, "workspace must not overlap xq"),
])
def test_gated_linear_backward_refuses(over, code, needle):
    assert call("moe_gated_linear_backward", L.GatedLinearBackwardArgs, GBWD, **over) == code
    assert needle in M.moe_last_error() and "moe_gated_linear_backward" in M.moe_last_error()


LORA = dict(T=6, K=72, N=48, R=24, num_adapters=3, num_seqs=2, x=at(0), ld_x=80, a=at(1), b=at(2), scale=at(3), adapter_ids=at(4),
            seq_offsets=at(5), residual=at(6), ld_residual=48, y=at(7), ld_y=48, out_dtype=1, workspace=at(8), workspace_bytes=1 << 20)


@pytest.mark.parametrize("over,code,needle", [
    (dict(T=0), B.MOE_ERR_INVALID, "T, K, N, R"), (dict(R=0), B.MOE_ERR_INVALID, "T, K, N, R"), (dict(K=70), B.MOE_ERR_UNSUPPORTED, "multiples of 8"),
    (dict(R=12), B.MOE_ERR_UNSUPPORTED, "multiples of 8"), (dict(N=40), B.MOE_ERR_UNSUPPORTED, "of 16"), (dict(R=264), B.MOE_ERR_UNSUPPORTED, "256"),
    (dict(K=65544, ld_x=65544), B.MOE_ERR_UNSUPPORTED, "65536"), (dict(num_adapters=0), B.MOE_ERR_INVALID, "num_adapters"),
    (dict(num_seqs=0), B.MOE_ERR_INVALID, "num_seqs"), (dict(seq_offsets=None), B.MOE_ERR_INVALID, "must be T"),
    (dict(num_seqs=(1 << 20) + 1), B.MOE_ERR_UNSUPPORTED, "num_seqs"), (dict(T=(1 << 23) + 1), B.MOE_ERR_UNSUPPORTED, "T ("),
    (dict(adapter_ids=None), B.MOE_ERR_INVALID, "adapter_ids"), (dict(out_dtype=3), B.MOE_ERR_INVALID, "out_dtype"),
    (dict(ld_x=64), B.MOE_ERR_INVALID, "ld_x"), (dict(ld_x=(1 << 24) + 8), B.MOE_ERR_UNSUPPORTED, "ld_x"), (dict(ld_y=40), B.MOE_ERR_INVALID, "ld_y"), (dict(ld_residual=8), B.MOE_ERR_INVALID, "ld_residual"),
    (dict(ld_x=76), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(b=at(2, 8)), B.MOE_ERR_UNSUPPORTED, "aligned"), (dict(y=at(7, 2)), B.MOE_ERR_UNSUPPORTED, "aligned"),
    (dict(scale=at(3, 2)), B.MOE_ERR_INVALID, "scale"), (dict(adapter_ids=at(4, 1)), B.MOE_ERR_INVALID, "adapter_ids"), (dict(seq_offsets=at(5, 2)), B.MOE_ERR_INVALID, "seq_offsets"),
    (dict(workspace=None), B.MOE_ERR_WORKSPACE, "workspace"), (dict(workspace_bytes=100), B.MOE_ERR_WORKSPACE, "need"),
    (dict(workspace=at(8, 64)), B.MOE_ERR_INVALID, "256-byte"), (dict(y=at(0)), B.MOE_ERR_INVALID, "y must not overlap x"),
    (dict(y=at(2)), B.MOE_ERR_INVALID, "y must not overlap b"), (dict(y=at(6, 16)), B.MOE_ERR_INVALID, "residual"),
    (dict(y=at(6), ld_y=56), B.MOE_ERR_INVALID, "residual"), (dict(workspace=at(6)), B.MOE_ERR_INVALID, "workspace must not overlap residual"),
    (dict(workspace=at(7)), B.MOE_ERR_INVALID, "y and workspace"), (dict(workspace=at(1)), B.MOE_ERR_INVALID, "workspace must not overlap a"),
])
def test_lora_refuses(over, code, needle):
    assert call("moe_lora", L.LoraArgs, LORA, **over) == code
    assert needle in M.moe_last_error() and "moe_lora" in M.moe_last_error()
