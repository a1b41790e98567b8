"""The norms' gradients where none comes through x, although the forward call took it."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import step_ref as step
from tests import test_gpu_norm as norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [64, 777, 1031, 2048, 8192, 8200])
@pytest.mark.parametrize("post", [True, False])
def test_a_row_of_zeros_without_eps(H, post):
    """Its s1 is infinite, x not a number; neither has a part in the gradient by r'."""
    c = norm._case(9, H, "bf16", "fp32", post, True)
    c["resid"][4] = 0
    c["gate"][4] = 0
    r2, _, rstd = norm._forward(c, post, "bf16", "fp32", eps=0.0)
    assert (r2[4] == 0).all() and torch.isinf(rstd[4, 1]) and torch.isfinite(rstd[:, 0]).all()
    o = dict(dresid=torch.empty_like(c["resid"]), df=torch.empty_like(c["f"]), dgate=torch.empty(9, device="cuda"))
    if post:
        o["dw_post"] = torch.empty(H, device="cuda")
    q.moe_norm_residual_bwd(r2, rstd, q.make_norm_workspace(H), dresid_out=c["dr2"], f=c["f"], w_post=c["w_post"],
                            gate=c["gate"], post_norm=post, alpha=norm.ALPHA, beta=norm.BETA, **o)
    d = [c[n].double() for n in ("dr2", "f", "gate")]
    w = None if c["w_post"] is None else c["w_post"].double()
    want = step.norm_back(None, d[0], d[1], r2.double(), w, None, d[2], rstd[:, :1].double(), None, post,
                          norm.ALPHA, norm.BETA)
    for n, t in o.items():
        step.near(t, *want[n], what=n)
