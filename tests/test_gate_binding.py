"""What the gate's and the projection's binding refuses beyond test_gate_abi.py (no GPU)."""
import pytest
import torch

import top_routing_expert_warp_b200 as moe
from test_gate_abi import OnDevice
from top_routing_expert_warp_b200 import build as moe_build


@pytest.mark.parametrize("code", [2, 7, -1])
def test_binding_refuses_unknown_element_types(code):
    """A configuration with an element type that does not exist is an invalid argument, as in C."""
    moe_build.build()
    ws = OnDevice(torch.zeros(1 << 16, dtype=torch.uint8))
    l, idx, w = (OnDevice(t) for t in (torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)))
    cfg = moe.make_route_config(4, 8, 2)
    cfg.dtype = code
    with pytest.raises(moe.MoeError) as err:
        moe.moe_route(cfg, l, None, idx, w, None, ws)
    assert err.value.status == moe.MOE_ERR_INVALID_ARG
    lc = moe.make_linear_config(4, 8, 3)
    lc.out_dtype = code
    x, W, y = (OnDevice(torch.zeros(*s).bfloat16()) for s in ((4, 8), (3, 8), (4, 3)))
    with pytest.raises(moe.MoeError) as err:
        moe.moe_linear(lc, x, W, None, None, y, None, ws)
    assert err.value.status == moe.MOE_ERR_INVALID_ARG
