"""Edges of the operators around the expert step that need no GPU."""
import pytest

import mixture_experts_fp8_amd as M
from mixture_experts_fp8_amd import binding as B
from mixture_experts_fp8_amd import layer as L

from test_layer_abi import BAL, CB, RB, _route, at, call


@pytest.mark.parametrize("over,needle", [(dict(clear_rows=2), "clear_rows"), (dict(clear_rows=-1), "clear_rows"),
                                         (dict(clear_rows=1, dexpert_out=at(1)), "dexpert_out must not overlap expert_out")])
def test_combine_backward_refuses_clear_rows(over, needle):
    # cleared rows of expert_out itself may be ones that the weights' gradient still reads
    assert call("moe_combine_backward", L.CombineBackwardArgs, CB, **over) == B.MOE_ERR_INVALID
    assert needle in M.moe_last_error()


@pytest.mark.parametrize("name,i", [("topk_ids", 1), ("losses", 3), ("counts", 4), ("mean_probs", 5), ("seq_offsets", 2)])
@pytest.mark.parametrize("off", [1, 2])
def test_balance_loss_refuses_unaligned(name, i, off):
    assert call("moe_balance_loss", L.BalanceLossArgs, dict(BAL, route=_route()), **{name: at(i, off)}) == B.MOE_ERR_INVALID
    assert name in M.moe_last_error() and "aligned" in M.moe_last_error()


@pytest.mark.parametrize("name,i", [("topk_ids", 1), ("dtopk_weights", 2), ("counts", 3), ("dlogits", 5)])
@pytest.mark.parametrize("off", [1, 2])
def test_route_backward_refuses_unaligned(name, i, off):
    assert call("moe_route_backward", L.RouteBackwardArgs, dict(RB, route=_route()), **{name: at(i, off)}) == B.MOE_ERR_INVALID
    assert name in M.moe_last_error() and "aligned" in M.moe_last_error()


@pytest.mark.parametrize("name,i", [("assign_pos", 2), ("topk_weights", 3), ("dtopk_weights", 4)])
@pytest.mark.parametrize("off", [1, 2])
def test_combine_backward_refuses_unaligned(name, i, off):
    assert call("moe_combine_backward", L.CombineBackwardArgs, CB, **{name: at(i, off)}) == B.MOE_ERR_INVALID
    assert name in M.moe_last_error() and "aligned" in M.moe_last_error()
