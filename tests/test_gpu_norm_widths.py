"""The norms around a block on both sides of every width at which the kernel
changes, forward and backward, and the grids of rows that start within a four."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import test_gpu_norm as norm

pytestmark = pytest.mark.gpu

# forward 2^n | 2^n + 1; backward 2^n | 2^n + 4, and 2^n - 3 | 2^n - 2 for rows that are no whole fours
ODD = [n + d for n in (256, 512, 1024, 2048, 4096, 8192) for d in (-3, -2, -1, 1)] + [777, 16383, 16385]
FOURS = [n + d for n in (256, 512, 1024, 2048, 4096, 8192, 16384) for d in (0, 4)]


def _both_ways(T, H, dtype, resid):
    c = norm._case(T, H, dtype, resid, True, True)
    r2, x, rstd = norm._forward(c, True, dtype, resid)
    norm._check_forward(c, True, r2, x, rstd, what=f"{T}x{H}")
    got = norm._backward(c, True, r2, rstd, q.make_norm_workspace(H))
    norm._check_backward(c, True, r2, rstd, got, f"{T}x{H}")
    place = c["dr2"].clone()
    q.moe_norm_residual_bwd(r2, rstd, dx=c["dx"], dresid_out=place, f=c["f"], w_pre=c["w_pre"], w_post=c["w_post"],
                            gate=c["gate"], post_norm=True, alpha=norm.ALPHA, beta=norm.BETA, dresid=place)
    assert torch.equal(place, got["dresid"])


@pytest.mark.parametrize("dtype,resid", [("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("H", ODD + FOURS)
def test_both_sides_of_a_width(H, dtype, resid):
    _both_ways(6, H, dtype, resid)


@pytest.mark.parametrize("H", [101, 301, 510, 777, 1021])
@pytest.mark.parametrize("per_sm", [2, 4, 8, 16])
@pytest.mark.parametrize("more", [-1, 0, 1, 3])
def test_rows_around_a_whole_grid(H, per_sm, more):
    """One row a thread and more, with eight, four and two rows a block."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    _both_ways(per_sm * sms + more, H, "bf16", "fp32")
