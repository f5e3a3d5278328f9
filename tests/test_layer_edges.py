"""Edges of the operators around the expert step that need no GPU."""
import pytest

import mixture_experts_fp8_amd as M
from mixture_experts_fp8_amd import binding as B
from mixture_experts_fp8_amd import layer as L

from test_layer_abi import CB, at, call


@pytest.mark.parametrize("over,needle", [(dict(clear_rows=2), "clear_rows"), (dict(clear_rows=-1), "clear_rows"),
                                         (dict(clear_rows=1, dexpert_out=at(1)), "dexpert_out must not overlap expert_out")])
def test_combine_backward_refuses_clear_rows(over, needle):
    # cleared rows of expert_out itself may be ones that the weights' gradient still reads
    assert call("moe_combine_backward", L.CombineBackwardArgs, CB, **over) == B.MOE_ERR_INVALID
    assert needle in M.moe_last_error()
