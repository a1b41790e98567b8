"""The sigmoid of the SwiGLU epilogues: off by at most 7 + 1.2 |g| steps of 2^-23.
The outputs have 16 bits, so it is looked at across their borders: factors that put
the exact product just further from the middle of two outputs than that error and
the products' two roundings (one step) have to come out on their own side."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q

pytestmark = pytest.mark.gpu

N = 20001                                    # gates


def _split(v):
    """fp32 values as the sum of three in bf16, exactly."""
    parts = []
    for _ in range(3):
        parts.append(v.bfloat16())
        v = v - parts[-1].float()
    assert (v == 0).all()
    return parts


def _factors(a, steps, seed):
    """fp32 factors u with a u above (first half) or below a middle of two bf16 values, by `steps` of 2^-23."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    odd = torch.randint(128, 256, a.shape, generator=gen, device="cuda").double() + 0.5     # 9 bits: a middle
    side = torch.where(torch.arange(a.numel(), device="cuda") % 2 == 0, 1.0, -1.0).double()
    # the rounding of u to fp32 may take half a step back
    u = (odd / a * (1 + side * (steps + 1) * 2.0 ** -23)).float()
    exact = a * u.double()
    assert ((exact - odd) * side >= odd * steps * 2.0 ** -23).all()
    return u, torch.where(side > 0, torch.ceil(odd), torch.floor(odd))


def _gates():
    """From -60 to 60, and near zero."""
    g = torch.linspace(-60.0, 60.0, N, device="cuda")
    g[::5] = torch.linspace(-2.0, 2.0, g[::5].numel(), device="cuda")
    return torch.where(g.abs() < 2.0 ** -10, 2.0 ** -10, g)


def test_forward():
    g = _gates()
    a = g.double() * torch.sigmoid(g.double())
    u, want = _factors(a, 8 + 1.2 * g.double().abs(), 3)
    w = torch.zeros(1, 2 * N, 8, dtype=torch.bfloat16, device="cuda")
    for i, (x, y) in enumerate(zip(_split(g), _split(u))):
        w[0, 0::2, i], w[0, 1::2, i] = x, y
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    x[:, :3] = 1
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    h = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    q.moe_grouped_swiglu(x, w, off, h, q.make_grouped_workspace())
    assert torch.equal(h[0].double(), want)


def test_backward():
    g = _gates().bfloat16()
    a = g.double() * torch.sigmoid(g.double())
    dh, want = _factors(a, 8 + 1.2 * g.double().abs(), 5)
    w = torch.stack(_split(dh))[None].contiguous()
    dy = torch.ones(1, 3, dtype=torch.bfloat16, device="cuda")
    p = torch.stack([g, torch.ones_like(g)], dim=1).reshape(1, 2 * N).contiguous()
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    dp = torch.empty_like(p)
    q.moe_grouped_swiglu_bwd(dy, w, p, off, dp, q.make_grouped_workspace())
    assert torch.equal(dp[0, 1::2].double(), want)
