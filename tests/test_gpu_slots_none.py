"""Tokens whose slots have no rows at all: every slot is out of range."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [64, 2048, 1031])
def test_no_slots(H):
    dout = torch.ones(5, H, dtype=torch.bfloat16, device="cuda")
    inv = torch.arange(10, dtype=torch.int32, device="cuda")
    none, w = torch.empty(0, H, dtype=torch.bfloat16, device="cuda"), torch.ones(5, 2, device="cuda")
    ws, dw = q.make_grouped_workspace(), torch.full((5, 2), 7.0, device="cuda")
    q.moe_slots_spread(dout, inv, ws, dy=none, weights=w, y=none, dweights=dw)
    assert (dw == 0).all() and q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
    q.moe_slots_spread(dout, inv, ws, dy=none)
    assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
    out = torch.full_like(dout, 7.0)
    q.moe_slots_combine(none, inv, out, ws, weights=w)
    assert (out == 0).all() and q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
