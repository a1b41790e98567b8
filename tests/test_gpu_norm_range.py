"""The norms' gradients for rows of any magnitude whose sum of squares fp32 holds."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import step_ref as step

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# every kernel: one warp a row to sixteen, rows that start within a four, rows read once a pass
WIDTHS = [8, 264, 520, 777, 1031, 2048, 4099, 8192, 8200, 16389]
SIZES = [(1e-17, 1e-17), (1e-17, 1e17), (1e-13, 1.0), (1.0, 1e-13), (1e13, 1.0), (1.0, 1e13), (1e15, 1e15), (1e17, 1.0),
         (1e17, 1e-17), (1e17, 1e17)]
ALPHA, BETA = 0.875, 1.25


def _backward(T, H, dtype, resid, r_size, f_size, post, dx_size=1.0):
    """Gradients of rows r' and f of root mean squares r_size and f_size, their norms without eps."""
    g = torch.Generator(device="cuda").manual_seed(T + H)

    def draw(*s, scale=1.0, dt="fp32"):
        return (scale * torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)).to(DT[dt])
    f, r2, dx = draw(T, H, scale=f_size, dt=dtype), draw(T, H, scale=r_size, dt=resid), draw(T, H, scale=dx_size, dt=dtype)
    dr2 = draw(T, H, scale=dx_size / r_size, dt=resid)      # as large as x's part of the gradient
    w_pre, w_post = 1 + draw(H, scale=0.2), 1 + draw(H, scale=0.2) if post else None
    gate = torch.sigmoid(draw(T))
    rstd = torch.ones(T, 2, device="cuda")
    rstd[:, 1] = r2.double().square().mean(dim=1).rsqrt()
    if post:
        rstd[:, 0] = f.double().square().mean(dim=1).rsqrt()
    o = dict(dresid=torch.empty_like(r2), df=torch.empty_like(f), dgate=torch.empty(T, device="cuda"),
             dw_pre=torch.empty(H, device="cuda"))
    if post:
        o["dw_post"] = torch.empty(H, device="cuda")
    q.moe_norm_residual_bwd(r2, rstd, q.make_norm_workspace(H), dx=dx, dresid_out=dr2, f=f, w_pre=w_pre, w_post=w_post,
                            gate=gate, post_norm=post, alpha=ALPHA, beta=BETA, **o)
    d = [None if t is None else t.double() for t in (dx, dr2, f, r2, w_post, w_pre, gate, rstd)]
    want = step.norm_back(*d[:7], *d[7].split(1, dim=1), post, ALPHA, BETA)
    for n, t in o.items():
        v, err = want[n]
        # what the type cannot hold: a gradient of 1e16 in fp16, whose largest value is 65504
        over = v.abs() > 2 * torch.finfo(t.dtype).max
        assert torch.equal(t[over].double(), v[over].sign() * float("inf"))
        step.near(t[~over], v[~over], err[~over], what=n)


@pytest.mark.parametrize("r_size,f_size", SIZES)
@pytest.mark.parametrize("H", WIDTHS)
def test_backward_of_rows_of_any_size(H, r_size, f_size):
    _backward(5, H, "bf16", "fp32", r_size, f_size, True)


@pytest.mark.parametrize("H", [520, 2048, 8200])
@pytest.mark.parametrize("dtype,resid,r_size,post", [("bf16", "bf16", 1e15, True), ("bf16", "bf16", 1e-15, False),
                                                     ("fp16", "fp32", 1e16, True), ("fp16", "fp32", 1e-16, False)])
def test_backward_of_rows_of_any_size_in_other_types(H, dtype, resid, r_size, post):
    _backward(300, H, dtype, resid, r_size, 1.0, post)


@pytest.mark.parametrize("H", [777, 2048, 8200])
def test_backward_of_large_rows_and_small_gradients(H):
    """s1^2 times the mean leaves fp32's normal values where s1 times it does not."""
    _backward(5, H, "bf16", "fp32", 1e17, 1.0, True, dx_size=1e-5)
