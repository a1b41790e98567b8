"""The norms around a block with its gate and the residual, forward and backward,
against 64-bit plain forms."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import step_ref as step

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TYPES = [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "fp16")]
SHAPES = [(1, 1), (1, 2048), (5, 8), (3, 37), (40, 64), (9, 264), (300, 512), (33, 1000), (17, 1031), (700, 1024),
          (21, 1032), (160, 2048), (35, 2056), (19, 4096), (11, 8192), (7, 8200), (3, 16384), (2, 16392), (4, 20001)]
ALPHA, BETA, EPS = 0.875, 1.25, 1e-5


def _case(T, H, dtype, resid, post, gated, weights=True):
    g = torch.Generator(device="cuda").manual_seed(T + H)

    def draw(*s, scale=1.0, dt="fp32"):
        return (scale * torch.randn(*s, generator=g, device="cuda")).to(DT[dt])
    return dict(f=draw(T, H, scale=0.5, dt=dtype), resid=draw(T, H, scale=3.0, dt=resid),
                w_pre=1 + draw(H, scale=0.2) if weights else None,
                w_post=1 + draw(H, scale=0.2) if weights and post else None,
                gate=torch.sigmoid(draw(T)) if gated else None, dx=draw(T, H, dt=dtype), dr2=draw(T, H, dt=resid))


def _d(t):
    return None if t is None else t.double()


def _check_forward(c, post, r2, x, rstd, alpha=ALPHA, beta=BETA, eps=EPS, what=""):
    want, err, s0 = step.norm(_d(c["f"]), _d(c["resid"]), _d(c["w_post"]), _d(c["gate"]), post, alpha, beta, eps)
    step.near(r2, want, err, what + " r'")
    want, err, s1 = step.pre(r2.double(), _d(c["w_pre"]), eps)
    step.near(x, want, err, what + " x")
    n = (step.depth(r2.shape[1]) / 2 + 6) * step.U
    step.near(rstd[:, :1], s0, n * s0)
    step.near(rstd[:, 1:], s1, n * s1)


def _forward(c, post, dtype, resid, **kw):
    T, H = c["f"].shape
    r2, x = torch.full((T, H), 7.0, dtype=DT[resid], device="cuda"), torch.full((T, H), 7.0, dtype=DT[dtype], device="cuda")
    rstd = torch.empty(T, 2, device="cuda")
    args = dict(alpha=ALPHA, beta=BETA, eps=EPS) | kw
    q.moe_norm_residual(c["resid"], r2, f=c["f"], x=x, w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"],
                        post_norm=post, rstd=rstd, **args)
    return r2, x, rstd


@pytest.mark.parametrize("post,gated", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype,resid", TYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, dtype, resid, post, gated):
    c = _case(T, H, dtype, resid, post, gated)
    r2, x, rstd = _forward(c, post, dtype, resid)
    _check_forward(c, post, r2, x, rstd, what=f"{T}x{H}")
    # in place, each output alone
    place, alone = c["resid"].clone(), torch.empty_like(x)
    kw = dict(f=c["f"], w_post=c["w_post"], gate=c["gate"], post_norm=post, alpha=ALPHA, beta=BETA, eps=EPS)
    q.moe_norm_residual(place, place, **kw)
    q.moe_norm_residual(c["resid"], x=alone, w_pre=c["w_pre"], **kw)
    assert torch.equal(place, r2) and torch.equal(alone, x)


@pytest.mark.parametrize("dtype,resid", TYPES)
@pytest.mark.parametrize("T,H", [(1, 2048), (40, 64), (17, 1031), (35, 2056), (11, 8192)])
def test_norm_alone_and_unit_weights(T, H, dtype, resid):
    """Without a branch it is the norm before a block: fp32 rows as moe_rmsnorm takes them."""
    c = _case(T, H, dtype, resid, False, False, weights=False)
    x, rstd = torch.empty(T, H, dtype=DT[dtype], device="cuda"), torch.empty(T, 2, device="cuda")
    q.moe_norm_residual(c["resid"], x=x, rstd=rstd, eps=EPS)
    want, err, _ = step.pre(c["resid"].double(), None, EPS)
    step.near(x, want, err)
    assert (rstd[:, 0] == 1).all()
    if (resid, dtype, H) == ("fp32", "bf16", 2048):      # a width that moe_rmsnorm takes
        old = torch.empty_like(x)
        q.moe_rmsnorm(c["resid"], old, eps=EPS)
        step.near(old, want, err)


def _backward(c, post, r2, rstd, ws, **kw):
    T, H = c["f"].shape
    o = dict(dresid=torch.full_like(c["resid"], 7.0), df=torch.full_like(c["f"], 7.0),
             dw_pre=torch.full((H,), 7.0, device="cuda"))
    if c["gate"] is not None:
        o["dgate"] = torch.full((T,), 7.0, device="cuda")
    if post:
        o["dw_post"] = torch.full((H,), 7.0, device="cuda")
    o |= kw
    q.moe_norm_residual_bwd(r2, rstd, ws, dx=c["dx"], dresid_out=c["dr2"], f=c["f"], w_pre=c["w_pre"],
                            w_post=c["w_post"], gate=c["gate"], post_norm=post, alpha=ALPHA, beta=BETA, **o)
    return o


def _check_backward(c, post, r2, rstd, got, what="", dx=True, dr2=True):
    want = step.norm_back(_d(c["dx"]) if dx else None, _d(c["dr2"]) if dr2 else None, _d(c["f"]), _d(r2),
                          _d(c["w_post"]), _d(c["w_pre"]), _d(c["gate"]), *_d(rstd).split(1, dim=1), post, ALPHA, BETA)
    for n, t in got.items():
        if t is not None:
            step.near(t, *want[n], what=f"{what} {n}")


@pytest.mark.parametrize("post,gated", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype,resid", TYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(T, H, dtype, resid, post, gated):
    c = _case(T, H, dtype, resid, post, gated)
    r2, _, rstd = _forward(c, post, dtype, resid)
    ws = q.make_norm_workspace(H)
    ws.fill_(255)                                # NaN patterns: whatever it held is not used
    got = _backward(c, post, r2, rstd, ws)
    _check_backward(c, post, r2, rstd, got, f"{T}x{H}")
    again = _backward(c, post, r2, rstd, ws)
    assert all(torch.equal(got[n], again[n]) for n in got)
    # the residual's gradient in place; without the weights' gradients, which alone need the workspace
    place = c["dr2"].clone()
    q.moe_norm_residual_bwd(r2, rstd, dx=c["dx"], dresid_out=place, f=c["f"], w_pre=c["w_pre"],
                            w_post=c["w_post"], gate=c["gate"], post_norm=post, alpha=ALPHA, beta=BETA, dresid=place)
    assert torch.equal(place, got["dresid"])


@pytest.mark.parametrize("dx,dr2", [(True, False), (False, True)])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("T,H", [(1, 2048), (40, 64), (17, 1031), (35, 2056), (11, 8192), (700, 520)])
def test_backward_from_one_side(T, H, post, dx, dr2):
    c = _case(T, H, "bf16", "fp32", post, True)
    if not dx:
        c["w_pre"] = None
    r2, _, rstd = _forward(c, post, "bf16", "fp32")
    o = dict(dresid=torch.empty_like(c["resid"]), df=torch.empty_like(c["f"]), dgate=torch.empty(T, device="cuda"),
             dw_pre=torch.empty(H, device="cuda") if dx else None,
             dw_post=torch.empty(H, device="cuda") if post else None)
    q.moe_norm_residual_bwd(r2, rstd, q.make_norm_workspace(H), dx=c["dx"] if dx else None,
                            dresid_out=c["dr2"] if dr2 else None, f=c["f"], w_pre=c["w_pre"], w_post=c["w_post"],
                            gate=c["gate"], post_norm=post, alpha=ALPHA, beta=BETA, **o)
    _check_backward(c, post, r2, rstd, o, dx=dx, dr2=dr2)


def test_backward_of_the_norm_alone():
    c = _case(50, 776, "fp16", "fp32", False, False)
    rstd, x = torch.empty(50, 2, device="cuda"), torch.empty_like(c["f"])
    q.moe_norm_residual(c["resid"], x=x, w_pre=c["w_pre"], rstd=rstd, eps=EPS)
    o = dict(dresid=torch.empty_like(c["resid"]), dw_pre=torch.empty(776, device="cuda"))
    q.moe_norm_residual_bwd(c["resid"], rstd, q.make_norm_workspace(776), dx=c["dx"], w_pre=c["w_pre"], **o)
    want = step.norm_back(_d(c["dx"]), None, None, _d(c["resid"]), None, _d(c["w_pre"]), None,
                          *_d(rstd).split(1, dim=1), False, 1.0, 1.0)
    for n in o:
        step.near(o[n], *want[n], what=n)


@pytest.mark.parametrize("T,H", [(40000, 64), (131072, 8), (20000, 520), (70000, 9)])
def test_long_column_sums_of_equal_terms(T, H):
    """Equal terms all round one way: added one by one, 2^17 of them come out 2e-3 off."""
    c = _case(T, H, "bf16", "fp32", True, False, weights=False)
    for n in ("f", "resid", "dx"):
        c[n].fill_(1.1)
    c["dr2"].fill_(0.3)
    r2, _, rstd = _forward(c, True, "bf16", "fp32")
    o = dict(dw_pre=torch.empty(H, device="cuda"), dw_post=torch.empty(H, device="cuda"))
    q.moe_norm_residual_bwd(r2, rstd, q.make_norm_workspace(H), dx=c["dx"], dresid_out=c["dr2"], f=c["f"],
                            post_norm=True, alpha=ALPHA, beta=BETA, **o)
    _check_backward(c, True, r2, rstd, o)


def test_zero_rows_and_infinities_stay_in_their_row():
    c = _case(12, 2048, "bf16", "fp32", True, True)
    c["f"][3], c["resid"][4], c["f"][5, 9], c["resid"][6, 8] = 0, 0, float("inf"), float("nan")
    c["f"][4] = 0
    r2, x, rstd = _forward(c, True, "bf16", "fp32")
    ok = [i for i in range(12) if i not in (5, 6)]
    _check_forward({k: (v[ok] if k in ("f", "resid", "gate") else v) for k, v in c.items()}, True, r2[ok], x[ok],
                   rstd[ok])
    assert torch.isnan(r2[5, 9]) and torch.isnan(x[6]).all() and (x[4] == 0).all()
    df = torch.empty_like(c["f"])
    q.moe_norm_residual_bwd(r2, rstd, dx=c["dx"], dresid_out=c["dr2"], f=c["f"], w_pre=c["w_pre"],
                            w_post=c["w_post"], gate=c["gate"], post_norm=True, df=df)
    assert torch.isfinite(df[ok]).all()


def test_no_rows():
    e, f32 = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, device="cuda")
    q.moe_norm_residual(e, e, f=e, x=e, rstd=f32)
    dw = [torch.full((64,), 5.0, device="cuda") for _ in range(2)]
    q.moe_norm_residual_bwd(e, f32, q.make_norm_workspace(64), dx=e, dresid_out=e, f=e, post_norm=True, dw_pre=dw[0],
                            dw_post=dw[1])
    assert (dw[0] == 0).all() and (dw[1] == 0).all()


@pytest.mark.parametrize("T,H", [(6, 2048), (500, 320), (4, 1031)])
def test_captured_on_another_stream(T, H):
    c = _case(T, H, "bf16", "fp32", True, True)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    r2, x, rstd = torch.empty_like(c["resid"]), torch.empty_like(c["f"]), torch.empty(T, 2, device="cuda")
    o = dict(dresid=torch.empty_like(c["resid"]), df=torch.empty_like(c["f"]), dgate=torch.empty(T, device="cuda"),
             dw_pre=torch.empty(H, device="cuda"), dw_post=torch.empty(H, device="cuda"))
    ws = q.make_norm_workspace(H)

    def once():
        q.moe_norm_residual(c["resid"], r2, f=c["f"], x=x, w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"],
                            post_norm=True, alpha=ALPHA, beta=BETA, eps=EPS, rstd=rstd)
        q.moe_norm_residual_bwd(r2, rstd, ws, dx=c["dx"], dresid_out=c["dr2"], f=c["f"], w_pre=c["w_pre"],
                                w_post=c["w_post"], gate=c["gate"], post_norm=True, alpha=ALPHA, beta=BETA, **o)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        once()
        with torch.cuda.graph(g, stream=s):
            once()
    torch.cuda.synchronize()
    c["f"].mul_(-0.5)
    c["gate"].mul_(0.25)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    _check_forward(c, True, r2, x, rstd)
    _check_backward(c, True, r2, rstd, o)


def test_binding_refuses():
    c = _case(4, 64, "bf16", "fp32", True, True)
    x = torch.empty_like(c["f"])
    with pytest.raises(TypeError, match="x must"):
        q.moe_norm_residual(c["resid"], f=c["f"], x=x.half())
    with pytest.raises(TypeError, match="residual"):
        q.moe_norm_residual(c["resid"].half(), x=x)
    with pytest.raises(ValueError, match="w_pre"):
        q.moe_norm_residual(c["resid"], x=x, w_pre=c["w_pre"].half())
    with pytest.raises(ValueError, match="shape"):
        q.moe_norm_residual(c["resid"], x=x[:3])
    with pytest.raises(ValueError, match="contiguous"):
        q.moe_norm_residual(c["resid"], x=torch.empty(64, 4, dtype=x.dtype, device="cuda").t())
    with pytest.raises(q.StrataError):
        q.moe_norm_residual(c["resid"], x=x, f=c["f"], w_post=c["w_post"])      # a weight of no norm
    with pytest.raises(q.StrataError):
        q.moe_norm_residual_bwd(c["resid"], torch.empty(4, 2, device="cuda"), dx=x, dw_pre=c["w_pre"])  # no workspace


@pytest.mark.parametrize("T", [150, 151, 152, 153, 303, 304, 305, 608, 611, 1217])
@pytest.mark.parametrize("H", [1029, 2501, 4099])
def test_backward_of_rows_that_start_within_a_four(T, H):
    """Around one row a thread and more, in grids that are cut to whole fours of rows."""
    c = _case(T, H, "bf16", "bf16", True, True)
    r2, _, rstd = _forward(c, True, "bf16", "bf16")
    got = _backward(c, True, r2, rstd, q.make_norm_workspace(H))
    _check_backward(c, True, r2, rstd, got, f"{T}x{H}")
