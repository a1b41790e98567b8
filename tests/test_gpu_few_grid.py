"""The few-row products around a grid of one block an SM, where their kernel changes."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import grouped_ref as ref
from tests import step_ref as step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [264, 8200])                   # short and long reductions
@pytest.mark.parametrize("counts", [[1], [0, 5, 3, 0]], ids=str)
@pytest.mark.parametrize("more", [-4, -2, 0, 2, 4])
def test_around_a_block_an_sm(more, counts, K, dtype):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    M, E = sum(counts), len(counts)
    N = sms * 8 * 4 // min(M, E) + more                      # eight warps a block, four rows of W each
    g = torch.Generator(device="cuda").manual_seed(N + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    w = (K ** -0.5 * torch.randn(E, N, K, generator=g, device="cuda")).to(dtype)
    off, ws = ref.offsets_of(counts).cuda(), q.make_grouped_workspace()
    y, y32 = torch.empty(M, N, dtype=dtype, device="cuda"), torch.empty(M, N, device="cuda")
    h, p = torch.empty(M, N // 2, dtype=dtype, device="cuda"), torch.empty_like(y)
    q.moe_grouped_mm(x, w, off, y, ws)
    q.moe_grouped_mm(x, w, off, y32, ws)
    q.moe_grouped_swiglu(x, w, off, h, ws, p=p)
    want, mags = ref.mm(x, w, off)
    for t in (y, y32, p):
        ref.check(t, want, mags, K)
    assert torch.equal(p, y)
    step.near(h, *step.swiglu(want, ref.sum_error(K, mags)))
    assert q.moe_get_device_status(ws) == q.STRATA_OK
