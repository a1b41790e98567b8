"""The weights' gradients of slots over long rows of equal terms, which all round
one way: added one by one, 8192 of a thread came out 1.2e-4 off."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import step_ref as step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,top_k", [(1, 1), (2, 5), (700, 1)])
@pytest.mark.parametrize("H", [2 ** 20 - 1, 2 ** 20 - 2, 2 ** 20 - 4, 2 ** 20, 65537])
def test_dweights_of_equal_terms(H, T, top_k, dtype):
    y = torch.full((T * top_k, H), 0.796875, dtype=dtype, device="cuda")
    dout = torch.full((T, H), 1.109375, dtype=dtype, device="cuda")
    inv = torch.randperm(T * top_k, device="cuda").int()
    ws, dw = q.make_grouped_workspace(), torch.empty(T, top_k, device="cuda")
    q.moe_slots_spread(dout, inv, ws, y=y, dweights=dw)
    # an access, the accesses of a piece, a thread's pieces (128 at most), a warp's threads, the warps
    depth = 8 + 64 + 128 + 5 + 4
    want = torch.full_like(dw, H * 0.796875 * 1.109375).double()
    step.near(dw, want, depth * step.U * want)
    assert q.moe_get_device_status(ws) == q.STRATA_OK
