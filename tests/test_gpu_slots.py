"""Slots combined into tokens and spread back, against 64-bit plain forms."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import step_ref as step

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# tokens, slots a token, width
SHAPES = [(1, 1, 1), (1, 8, 2048), (3, 2, 37), (16, 10, 2048), (251, 4, 1000), (70, 16, 264), (33, 3, 4104),
          (5, 5, 8193), (2, 9, 40000), (1000, 8, 64), (300, 6, 8), (9, 7, 12), (600, 8, 2048)]


def _case(T, K, H, dtype, spare=0):
    g = torch.Generator(device="cuda").manual_seed(T + K + H)
    M = T * K + spare

    def draw(*s):
        return torch.randn(*s, generator=g, device="cuda")
    inv = torch.randperm(M, generator=g, device="cuda")[:T * K].int().reshape(T, K)
    return draw(M, H).to(DT[dtype]), draw(T, H).to(DT[dtype]), inv, draw(T, K), q.make_grouped_workspace()


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
@pytest.mark.parametrize("T,K,H", SHAPES)
def test_combine(T, K, H, dtype, out):
    y, _, inv, w, ws = _case(T, K, H, dtype, spare=5)
    for weights in (w, None):
        o = torch.full((T, H), 7.0, dtype=DT[out], device="cuda")
        q.moe_slots_combine(y, inv.reshape(-1), o, ws, weights=weights)
        want, mag = step.combine(y, inv, weights)
        step.near(o, want, (K + 1) * step.U * mag)
    assert q.moe_get_device_status(ws) == q.STRATA_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,H", SHAPES)
def test_spread(T, K, H, dtype):
    y, dout, inv, w, ws = _case(T, K, H, dtype, spare=5)
    M = y.shape[0]
    want, there, dw, mag = step.spread(dout, inv, w, y, M)
    depth = H // 64 + 40                        # a thread's terms, then the threads
    dy, got = torch.full_like(y, 7.0), torch.full((T, K), 7.0, device="cuda")
    q.moe_slots_spread(dout, inv, ws, dy=dy, weights=w, y=y, dweights=got)
    step.near(dy[there], want[there], step.U * want[there].abs())
    assert (dy[~there] == 7).all()
    step.near(got, dw, depth * step.U * mag)
    # each output alone, and the gather
    alone, dw_alone = torch.full_like(y, 7.0), torch.empty_like(got)
    q.moe_slots_spread(dout, inv, ws, dy=alone, weights=w)
    q.moe_slots_spread(dout, inv, ws, weights=w, y=y, dweights=dw_alone)
    assert torch.equal(alone, dy) and torch.equal(dw_alone, got)
    q.moe_slots_spread(dout, inv, ws, dy=alone)
    assert torch.equal(alone[inv.long().reshape(-1)], dout.repeat_interleave(K, dim=0))
    assert q.moe_get_device_status(ws) == q.STRATA_OK


@pytest.mark.parametrize("H", [64, 37, 2056])
def test_bad_slots_are_left_out(H):
    y, dout, inv, w, _ = _case(4, 3, H, "bf16")
    inv[1, 2], inv[2, 0], inv[3] = -1, y.shape[0], torch.tensor([-2 ** 31, 2 ** 31 - 1, -7], device="cuda").int()
    ws = q.make_grouped_workspace()
    out = torch.full((4, H), 7.0, dtype=torch.bfloat16, device="cuda")
    q.moe_slots_combine(y, inv, out, ws, weights=w)
    assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
    want, mag = step.combine(y, inv, w)
    step.near(out, want, 4 * step.U * mag)
    assert (out[3] == 0).all()
    dy, dw = torch.full_like(y, 7.0), torch.full((4, 3), 7.0, device="cuda")
    q.moe_slots_spread(dout, inv, ws, dy=dy, weights=w, y=y, dweights=dw)
    assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
    want, there, ref_dw, mag = step.spread(dout, inv, w, y, y.shape[0])
    step.near(dy[there], want[there], step.U * want[there].abs())
    assert (dy[~there] == 7).all()
    step.near(dw, ref_dw, 80 * step.U * mag)
    assert dw[1, 2] == 0 and dw[2, 0] == 0 and (dw[3] == 0).all()


def test_infinities_stay_in_their_token():
    y, dout, inv, w, ws = _case(8, 3, 72, "bf16")
    y[inv[2, 1].long(), 5], dout[4, 7] = float("inf"), float("nan")
    out, dw = torch.empty(8, 72, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 3, device="cuda")
    dy = torch.empty_like(y)
    q.moe_slots_combine(y, inv, out, ws, weights=w)
    q.moe_slots_spread(dout, inv, ws, dy=dy, weights=w, y=y, dweights=dw)
    bad = ~torch.isfinite(out)
    assert bad.sum() == 1 and bad[2, 5]
    bad = ~torch.isfinite(dw)
    assert bad.sum() == 4 and bad[4].all() and bad[2, 1]
    assert (~torch.isfinite(dy)).sum() == 3


def test_binding_refuses():
    y, dout, inv, w, ws = _case(4, 2, 64, "bf16")
    out = torch.empty_like(dout)
    with pytest.raises(ValueError, match="inv_perm"):
        q.moe_slots_combine(y, inv.long(), out, ws)
    with pytest.raises(ValueError, match="inv_perm"):
        q.moe_slots_combine(y, inv.reshape(-1)[:7].contiguous(), out, ws)
    with pytest.raises(ValueError, match="weights"):
        q.moe_slots_combine(y, inv, out, ws, weights=w.half())
    with pytest.raises(TypeError, match="out must"):
        q.moe_slots_combine(y, inv, out.half(), ws)
    with pytest.raises(ValueError, match="nothing"):
        q.moe_slots_spread(dout, inv, ws)
    with pytest.raises(TypeError, match="dy must"):
        q.moe_slots_spread(dout, inv, ws, dy=y.half())
    with pytest.raises(q.StrataError):
        q.moe_slots_spread(dout, inv, ws, dy=y, y=y)
    with pytest.raises(ValueError, match="contiguous"):
        q.moe_slots_combine(y.t().contiguous().t(), inv, out, ws)
