"""The tuning step's operators past 2^31 elements: rows at both ends and across the border, against
64-bit plain forms."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import grouped_ref as ref
from tests import step_ref as step

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _rows(M, width):
    """Rows at the start, around the element 2^31 and 2^32, and at the end."""
    at = [0, 1, 127, 128, M - 130, M - 2, M - 1] + [b // width + d for b in (2 ** 31, 2 ** 32) for d in (-1, 0, 1)]
    return torch.tensor(sorted({r for r in at if 0 <= r < M}), device="cuda")


def _rand(*s, scale=1.0, dtype=BF):
    t = torch.empty(*s, dtype=dtype, device="cuda")
    t.normal_(0, scale, generator=torch.Generator(device="cuda").manual_seed(sum(s)))
    return t


@pytest.mark.parametrize("K", [64, 37])
@pytest.mark.parametrize("keep8", [False, True])
def test_swiglu(K, keep8):
    M, I = 2 ** 21 + 77, 1024
    if K == 37:                       # on the CUDA cores: fewer rows, just past 2^31
        M = 2 ** 20 + 77
    x, w, wd = _rand(M, K), _rand(2, 2 * I, K, scale=K ** -0.5), _rand(2, K, I, scale=K ** -0.5)
    off = torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda")
    ws, rows = q.make_grouped_workspace(), _rows(M, 2 * I)
    group = (rows >= M // 3).long()
    h = torch.empty(M, I, dtype=BF, device="cuda")
    p = torch.empty(M, 2 * I, dtype=torch.uint8 if keep8 else BF, device="cuda")
    ps = torch.empty(M, 2 * I // 32, dtype=torch.uint8, device="cuda") if keep8 else None
    q.moe_grouped_swiglu(x, w, off, h, ws, p=p, p_scales=ps)
    want = torch.einsum("rk,rnk->rn", x[rows].double(), w[group].double())
    err = ref.sum_error(K, torch.einsum("rk,rnk->rn", x[rows].double().abs(), w[group].double().abs()))
    step.near(h[rows], *step.swiglu(want, err))
    if keep8:
        kept = torch.from_numpy(step.act8_load(p[rows].cpu().numpy(), ps[rows].cpu().numpy())).cuda()
        assert ((kept - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * want.abs().amax(dim=1, keepdim=True)).all()
    else:
        step.near(p[rows], want, err)
        kept = p[rows].double()
    dp = torch.empty(M, 2 * I, dtype=BF, device="cuda")
    q.moe_grouped_swiglu_bwd(x, wd, p, off, dp, ws, p_scales=ps, h=h)
    dh = torch.einsum("rk,rki->ri", x[rows].double(), wd[group].double())
    edh = ref.sum_error(K, torch.einsum("rk,rki->ri", x[rows].double().abs(), wd[group].double().abs()))
    (want, err), (h2, eh) = step.swiglu_back(dh, edh, kept)
    step.near(dp[rows], want, err)
    step.near(h[rows], h2, eh)
    assert q.moe_get_device_status(ws) == q.STRATA_OK


def test_act8():
    R, C = 2 ** 20 + 5, 2080
    x = _rand(R, C)
    codes, scales = (torch.empty(R, n, dtype=torch.uint8, device="cuda") for n in (C, C // 32))
    q.moe_act8_save(x, codes, scales)
    rows = _rows(R, C)
    want, byte = step.act8_save(x[rows].double().cpu().numpy())
    assert (codes[rows].cpu().numpy() == want).all() and (scales[rows].cpu().numpy() == byte).all()
    out, ws = torch.empty_like(x), q.make_grouped_workspace()
    perm = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    q.moe_act8_load(codes, scales, out, ws, perm=perm)
    vals = torch.from_numpy(step.act8_load(want, byte)).cuda().bfloat16()
    assert torch.equal(out[R - 1 - rows], vals)


@pytest.mark.parametrize("H", [2056, 2053])
def test_slots(H):
    T, K = 2 ** 18 + 3, 4
    M = T * K
    y, dout = _rand(M, H), _rand(T, H)
    inv = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda").reshape(T, K)
    w = _rand(T, K, dtype=torch.float32)
    ws, t = q.make_grouped_workspace(), torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    out, dw = torch.empty_like(dout), torch.empty(T, K, device="cuda")
    q.moe_slots_combine(y, inv, out, ws, weights=w)
    want, mag = step.combine(y[inv[t].long().reshape(-1)], torch.arange(5 * K, device="cuda").reshape(5, K), w[t])
    step.near(out[t], want, (K + 1) * step.U * mag)
    yt = y[inv[t].long().reshape(-1)].clone()
    q.moe_slots_spread(dout, inv, ws, dy=y, weights=w)
    q.moe_slots_spread(dout, inv, ws, weights=w, y=y, dweights=dw)
    want, _, _, _ = step.spread(dout[t], torch.arange(5 * K, device="cuda").reshape(5, K), w[t], None, 5 * K)
    got = y[inv[t].long().reshape(-1)]
    step.near(got, want, step.U * want.abs())
    assert not torch.equal(got, yt)
    _, _, want, mag = step.spread(dout[t], torch.arange(5 * K, device="cuda").reshape(5, K), w[t], got, 5 * K)
    step.near(dw[t], want, (H // 64 + 40) * step.U * mag)
    assert q.moe_get_device_status(ws) == q.STRATA_OK


@pytest.mark.parametrize("T,H", [(2 ** 20 + 3, 2052), (2 ** 18 + 3, 8200), (2 ** 23 + 5, 257)])
def test_norm(T, H):
    f, resid, dx = _rand(T, H, scale=0.5), _rand(T, H), _rand(T, H, scale=0.25)
    gate = torch.rand(T, device="cuda")
    r2, x, rstd = torch.empty_like(f), torch.empty_like(f), torch.empty(T, 2, device="cuda")
    q.moe_norm_residual(resid, r2, f=f, x=x, gate=gate, post_norm=True, rstd=rstd)
    t = _rows(T, H)
    want, err, s0 = step.norm(f[t].double(), resid[t].double(), None, gate[t].double(), True, 1.0, 1.0, 1e-6)
    step.near(r2[t], want, err)
    want, err, s1 = step.pre(r2[t].double(), None, 1e-6)
    step.near(x[t], want, err)
    dr2 = resid                                  # any gradient; taken in place
    had = dr2[t].double()
    dgate, dw = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
    q.moe_norm_residual_bwd(r2, rstd, q.make_norm_workspace(H), dx=dx, dresid_out=dr2, f=f, gate=gate,
                            post_norm=True, dresid=dr2, df=x, dgate=dgate, dw_pre=dw)
    want = step.norm_back(dx[t].double(), had, f[t].double(), r2[t].double(), None, None, gate[t].double(),
                          *rstd[t].double().split(1, dim=1), True, 1.0, 1.0)
    for got, name in ((dr2[t], "dresid"), (x[t], "df"), (dgate[t], "dgate")):
        step.near(got, *want[name], what=name)
    # the column sums, a slice of columns at a time
    for c in (0, H // 2, H - 8):
        cols = (dx[:, c:c + 8].double() * r2[:, c:c + 8].double() * rstd[:, 1:].double())
        step.near(dw[c:c + 8], cols.sum(dim=0), (640 + T // 4096 + 8) * step.U * cols.abs().sum(dim=0))
