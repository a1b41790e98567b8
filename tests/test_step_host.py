"""The tuning step's operators: argument checks (no GPU: all of them come before
any CUDA call), workspace sizes, and the plain forms' own pins."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from quantized_moe_expert_fwd_gb300 import build as qbuild
from tests import step_ref as step

P = 1 << 20          # an aligned address that no refused call reads
WS = 65536
MOST = 2 ** 31 - 1024
BIG = 2 ** 32 + 8    # passed on in 32 bits it would read as 8


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load()


def _swiglu(lib, dtype=0, x=P, w=P, M=4, K=64, I=32, E=2, off=P, h=P, p=0, ps=0, ws=P, n=WS):
    return lib.moe_grouped_swiglu(dtype, x, w, M, K, I, E, off, h, p, ps, ws, n, None)


def _swiglu_bwd(lib, dtype=0, x=P, w=P, p=P, ps=0, M=4, K=64, I=32, E=2, off=P, dp=P, h=0, ws=P, n=WS):
    return lib.moe_grouped_swiglu_bwd(dtype, x, w, p, ps, M, K, I, E, off, dp, h, ws, n, None)


BAD = [dict(dtype=2), dict(dtype=-1), dict(M=-1), dict(M=MOST + 1), dict(K=0), dict(K=(1 << 20) + 1), dict(I=0),
       dict(I=(1 << 19) + 1), dict(E=0), dict(E=1025), dict(x=0), dict(x=P + 8), dict(w=0), dict(w=P + 2),
       dict(off=0), dict(off=P + 2), dict(h=P + 4), dict(p=P + 8), dict(p=P, ps=P + 4), dict(p=P, ps=P, I=24),
       dict(ws=0), dict(ws=P + 16), dict(n=WS - 1)]


@pytest.mark.parametrize("kw", BAD + [dict(h=0), dict(ps=P)], ids=str)
def test_swiglu_refusals(lib, kw):
    assert _swiglu(lib, **kw) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", BAD + [dict(dp=0), dict(dp=P + 8), dict(p=0)], ids=str)
def test_swiglu_bwd_refusals(lib, kw):
    assert _swiglu_bwd(lib, **kw) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(x=0), dict(x=P + 8), dict(rows=-1),
                                dict(rows=MOST + 1), dict(cols=0), dict(cols=48), dict(cols=(1 << 20) + 32),
                                dict(codes=0), dict(codes=P + 8), dict(sc=0), dict(sc=P + 8)], ids=str)
def test_act8_save_refusals(lib, kw):
    a = dict(dtype=0, x=P, rows=4, cols=64, codes=P, sc=P) | kw
    assert lib.moe_act8_save(a["dtype"], a["x"], a["rows"], a["cols"], a["codes"], a["sc"],
                             None) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", [dict(codes=0), dict(sc=P + 8), dict(q_rows=-1), dict(q_rows=3), dict(cols=33),
                                dict(perm=P + 2), dict(top_k=0), dict(rows=-1), dict(od=3), dict(out=0),
                                dict(out=P + 4), dict(ws=0), dict(ws=P + 128), dict(n=8)], ids=str)
def test_act8_load_refusals(lib, kw):
    a = dict(codes=P, sc=P, q_rows=4, cols=64, perm=0, top_k=1, rows=4, od=0, out=P, ws=P, n=WS) | kw
    assert lib.moe_act8_load(a["codes"], a["sc"], a["q_rows"], a["cols"], a["perm"], a["top_k"], a["rows"],
                             a["od"], a["out"], a["ws"], a["n"], None) == q.STRATA_EINVAL


SLOTS = [dict(dtype=2), dict(M=-1), dict(H=0), dict(H=(1 << 20) + 1), dict(T=-1), dict(k=0), dict(k=17),
         dict(T=1 << 28, k=8), dict(inv=0), dict(inv=P + 2), dict(w=P + 1), dict(y=P + 8), dict(ws=0), dict(n=9)]


@pytest.mark.parametrize("kw", SLOTS + [dict(y=0), dict(od=1), dict(od=3), dict(out=0), dict(out=P + 8)], ids=str)
def test_slots_combine_refusals(lib, kw):
    a = dict(dtype=0, y=P, M=8, H=64, inv=P, w=P, T=4, k=2, od=0, out=P, ws=P, n=WS) | kw
    assert lib.moe_slots_combine(a["dtype"], a["y"], a["M"], a["H"], a["inv"], a["w"], a["T"], a["k"], a["od"],
                                 a["out"], a["ws"], a["n"], None) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", SLOTS + [dict(dout=0), dict(dout=P + 8), dict(dy=P + 4), dict(y=0), dict(dw=0),
                                        dict(dw=P + 2), dict(dy=0, dw=0, y=0)], ids=str)
def test_slots_spread_refusals(lib, kw):
    a = dict(dtype=0, dout=P, inv=P, w=P, y=P, T=4, k=2, M=8, H=64, dy=P, dw=P, ws=P, n=WS) | kw
    assert lib.moe_slots_spread(a["dtype"], a["dout"], a["inv"], a["w"], a["y"], a["T"], a["k"], a["M"], a["H"],
                                a["dy"], a["dw"], a["ws"], a["n"], None) == q.STRATA_EINVAL


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(rt=1), dict(rt=3), dict(T=-1), dict(T=MOST + 1), dict(H=0),
                                dict(H=(1 << 20) + 1), dict(f=0), dict(f=0, post=0), dict(f=P + 8), dict(r=0),
                                dict(r=P + 4), dict(post=0), dict(x=0), dict(r2=0, x=0, wpre=0), dict(x=P + 2),
                                dict(r2=P + 8), dict(wpost=P + 4), dict(wpre=P + 4), dict(gate=P + 2),
                                dict(rstd=P + 1), dict(alpha=NAN), dict(beta=INF), dict(eps=-1.0),
                                dict(eps=INF)], ids=str)
def test_norm_refusals(lib, kw):
    a = dict(dtype=0, rt=2, f=P, r=P, wpost=P, wpre=P, gate=P, T=4, H=64, post=1, alpha=1.0, beta=1.0, eps=1e-6,
             r2=P, x=P, rstd=P) | kw
    assert lib.moe_norm_residual(a["dtype"], a["rt"], a["f"], a["r"], a["wpost"], a["wpre"], a["gate"], a["T"],
                                 a["H"], a["post"], a["alpha"], a["beta"], a["eps"], a["r2"], a["x"], a["rstd"],
                                 None) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(rt=1), dict(T=-1), dict(H=0), dict(dx=0, dr2=0),
                                dict(dx=0, wpre=0), dict(dx=0, dwpre=0), dict(dx=P + 8), dict(dr2=P + 4),
                                dict(f=0), dict(f=P + 8), dict(r2=0), dict(post=0), dict(post=0, wpost=0),
                                dict(gate=0), dict(rstd=0), dict(df=P + 8), dict(dr=P + 8), dict(dgate=P + 2),
                                dict(dwpost=P + 4), dict(dwpre=P + 4), dict(ws=0), dict(ws=P + 16),
                                dict(n=WS + 64 * 4864 - 1), dict(alpha=INF), dict(beta=NAN),
                                dict(df=0, dr=0, dgate=0, dwpost=0, dwpre=0)], ids=str)
def test_norm_bwd_refusals(lib, kw):
    a = dict(dtype=0, rt=2, dx=P, dr2=P, f=P, r2=P, wpost=P, wpre=P, gate=P, rstd=P, T=4, H=64, post=1, alpha=1.0,
             beta=1.0, df=P, dr=P, dgate=P, dwpost=P, dwpre=P, ws=P, n=WS + 64 * 4864) | kw
    assert lib.moe_norm_residual_bwd(a["dtype"], a["rt"], a["dx"], a["dr2"], a["f"], a["r2"], a["wpost"],
                                     a["wpre"], a["gate"], a["rstd"], a["T"], a["H"], a["post"], a["alpha"],
                                     a["beta"], a["df"], a["dr"], a["dgate"], a["dwpost"], a["dwpre"], a["ws"],
                                     a["n"], None) == q.STRATA_EINVAL


def test_no_rows_launch_nothing(lib):
    assert _swiglu(lib, M=0, x=0, h=0, ws=0) == q.STRATA_OK
    assert _swiglu_bwd(lib, M=0, x=0, p=0, dp=0, ws=0) == q.STRATA_OK
    assert lib.moe_act8_save(0, None, 0, 64, None, None, None) == q.STRATA_OK
    assert lib.moe_act8_load(None, None, 0, 64, None, 1, 0, 0, None, None, 0, None) == q.STRATA_OK
    assert lib.moe_slots_combine(0, None, 0, 64, None, None, 0, 2, 0, None, None, 0, None) == q.STRATA_OK
    assert lib.moe_slots_spread(0, None, None, None, None, 0, 2, 0, 64, P, None, None, 0, None) == q.STRATA_OK
    assert lib.moe_norm_residual(0, 2, None, None, None, None, None, 0, 64, 0, 1.0, 1.0, 1e-6, P, None, None,
                                 None) == q.STRATA_OK


def test_norm_workspace_bytes(lib):
    assert q.moe_norm_workspace_bytes(1) == WS + 4864
    assert q.moe_norm_workspace_bytes(2048) == WS + 4864 * 2048
    for bad in (0, -1, (1 << 20) + 1, BIG):
        assert q.moe_norm_workspace_bytes(bad) == 0


def _meta(*shape, dtype=torch.bfloat16):
    """A tensor of that shape without memory."""
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_binding_refuses_sizes_past_32_bits(lib):
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    ws, off, inv = _meta(WS, dtype=u8), _meta(2, dtype=i32), _meta(8, dtype=i32)
    x, long = _meta(8, 32), _meta(BIG, 32)
    for call in (lambda: q.moe_grouped_swiglu(long, _meta(1, 64, 32), off, long, ws),
                 lambda: q.moe_grouped_swiglu(_meta(8, BIG), _meta(1, 64, BIG), off, x, ws),
                 lambda: q.moe_grouped_swiglu(x, _meta(1, BIG, 32), off, _meta(8, BIG // 2), ws),
                 lambda: q.moe_grouped_swiglu_bwd(long, _meta(1, 32, 32), _meta(BIG, 64), off, _meta(BIG, 64), ws),
                 lambda: q.moe_grouped_swiglu_bwd(x, _meta(1, 32, BIG // 2), x, off, x, ws),
                 lambda: q.moe_act8_save(long, _meta(BIG, 32, dtype=u8), _meta(BIG, 1, dtype=u8)),
                 lambda: q.moe_act8_load(_meta(8, 32, dtype=u8), _meta(8, 1, dtype=u8), x, ws, perm=inv, top_k=BIG),
                 lambda: q.moe_slots_combine(long, inv, x, ws),
                 lambda: q.moe_slots_spread(x, inv, ws, dy=long),
                 lambda: q.moe_norm_residual(_meta(BIG, 32, dtype=f32), x=long),
                 lambda: q.moe_norm_residual_bwd(_meta(8, BIG), _meta(8, 2, dtype=f32), dx=x)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_binding_takes_cuda_tensors_only(lib):
    x, u8 = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.uint8)
    off, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(WS, dtype=torch.uint8)
    for call in (lambda: q.moe_grouped_swiglu(x, torch.zeros(2, 64, 64, dtype=x.dtype), off, x[:, :32], ws),
                 lambda: q.moe_act8_save(x, u8, u8[:, :2]), lambda: q.moe_slots_combine(x, off, x, ws),
                 lambda: q.moe_norm_residual(x, x=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# --------------------------------------------------------- the plain forms
def test_plain_act8_hand_computed():
    x = np.zeros((1, 64))
    x[0, :8] = [448, -224, 1, 17, 18, 19, 2.0 ** -9, 1.4 * 2.0 ** -10]
    x[0, 32:36] = [449, 464, -480, 2.0 ** -10]
    codes, byte = step.act8_save(x)
    assert list(byte[0]) == [127, 128]                    # 448 2^0 holds 448, 449 takes the next
    v = step.act8_load(codes, byte)
    # between 16 and 32 the step is 2, ties to the even code; 2^-9 is the smallest value
    assert list(v[0, :8]) == [448, -224, 1, 16, 18, 20, 2.0 ** -9, 2.0 ** -9]
    assert list(v[0, 32:36]) == [448, 448, -480, 0]
    assert codes[0, 0] == 0x7e and codes[0, 1] == 0xf6
    x[0, 0], x[0, 40] = np.inf, np.nan
    codes, byte = step.act8_save(x)
    assert list(byte[0]) == [255, 255] and (codes == 0x7f).all() and np.isnan(step.act8_load(codes, byte)).all()
    tiny = np.full((1, 32), 2.0 ** -140)
    codes, byte = step.act8_save(tiny)
    assert byte[0, 0] == 1 and (codes == 0).all()
    assert step.act8_save(np.zeros((1, 32)))[1][0, 0] == 1


def _difference(fn, x, d, e=1e-6):
    return (fn(x + e * d) - fn(x - e * d)) / (2 * e)


def test_plain_swiglu_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    p, dh, d = (torch.randn(5, n, generator=g, dtype=torch.float64) * s for n, s in ((12, 4), (6, 1), (12, 1)))
    zero = torch.zeros_like(p)
    (dp, _), (h, _) = step.swiglu_back(dh, torch.zeros_like(dh), p)
    want = _difference(lambda v: (dh * step.swiglu(v, zero)[0]).sum(), p, d)
    assert abs((dp * d).sum() - want) < 1e-8 * (dp * d).abs().sum()
    assert torch.equal(h, step.swiglu(p, zero)[0])


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_plain_norm_gradients_against_differences(post, gated):
    gen = torch.Generator().manual_seed(5)

    def rnd(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)
    T, H, alpha, beta, eps = 4, 7, 0.7, 1.3, 1e-3
    v = dict(f=rnd(T, H), resid=rnd(T, H), w_post=rnd(H), w_pre=rnd(H), gate=rnd(T))
    dx, dr2 = rnd(T, H), rnd(T, H)

    def out(a):
        r2, _, s0 = step.norm(a["f"], a["resid"], a["w_post"] if post else None, a["gate"] if gated else None,
                              post, alpha, beta, eps)
        x, _, s1 = step.pre(r2, a["w_pre"], eps)
        return r2, x, s0, s1
    r2, x, s0, s1 = out(v)
    got = step.norm_back(dx, dr2, v["f"], r2, v["w_post"] if post else None, v["w_pre"],
                         v["gate"] if gated else None, s0, s1, post, alpha, beta)
    names = dict(f="df", resid="dresid", w_pre="dw_pre") | (dict(w_post="dw_post") if post else {}) \
        | (dict(gate="dgate") if gated else {})
    for name, grad in names.items():
        d = rnd(*v[name].shape)

        def loss(z):
            r2, x, _, _ = out(v | {name: z})
            return (dr2 * r2).sum() + (dx * x).sum()
        want = _difference(loss, v[name], d)
        assert abs((got[grad][0] * d).sum() - want) < 1e-7 * (1 + abs(want)), name


def test_plain_spread_is_the_gradient_of_combine():
    gen = torch.Generator().manual_seed(7)
    y, w = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((7, 5), (3, 2)))
    dout = torch.randn(3, 5, generator=gen, dtype=torch.float64)
    inv = torch.tensor([[4, 0], [6, -1], [2, 1]])
    dy, there, dw, _ = step.spread(dout, inv, w, y, 7)
    assert there.tolist() == [True, True, True, False, True, False, True] and dw[1, 1] == 0
    for d, grad, fn in ((torch.randn(7, 5, generator=gen, dtype=torch.float64), dy, lambda z: step.combine(z, inv, w)),
                        (torch.randn(3, 2, generator=gen, dtype=torch.float64), dw, lambda z: step.combine(y, inv, z))):
        want = _difference(lambda z: (dout * fn(z)[0]).sum(), y if grad is dy else w, d)
        assert abs((grad * d).sum() - want) < 1e-8
