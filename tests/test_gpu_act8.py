"""Rows kept in 8 bits, bit for bit against the definition."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import step_ref as step

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _save(x):
    R, C = x.shape
    codes = torch.full((R, C), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, C // 32), 0x55, dtype=torch.uint8, device="cuda")
    q.moe_act8_save(x, codes, scales)
    return codes, scales


def _same(x):
    codes, scales = _save(x)
    want, byte = step.act8_save(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(codes.cpu().numpy(), want)
    return codes, scales


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2048), (3, 96), (37, 160), (500, 2080), (4099, 64)])
def test_save(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-14, 9, (rows, 1), generator=g, device="cuda").float())
    _same(x.to(DT[dtype]))


def test_every_code_and_border():
    """Every e4m3 value, the middles between neighbours and the fp32 numbers next to those, with
    448 beside them to fix the scale; then the largest magnitudes next to the scales' borders."""
    t = torch.from_numpy(step.e4m3_table()).float()
    mid = (t[1:] + t[:-1]) / 2
    inf = torch.tensor(float("inf"))
    v = torch.cat([t, mid, torch.nextafter(mid, inf), torch.nextafter(mid, -inf)])
    v = torch.cat([v, -v, torch.zeros(-2 * v.numel() % 31)])
    x = torch.cat([torch.full((v.numel() // 31, 1), 448.0), v.reshape(-1, 31)], dim=1).cuda()
    for e in (0, -20, 100, -118):
        _same(x * 2.0 ** e)
    m = torch.tensor([448.0, 449.0, 447.0, 256.0, 255.5, 511.9])
    m = torch.cat([m, torch.nextafter(m, inf), torch.nextafter(m, -inf)])
    m = (m[:, None] * torch.exp2(torch.tensor([0.0, -30.0, 60.0, 118.0, -126.0, -130.0, -134.0, -140.0]))).reshape(-1, 1)
    _same((m * torch.linspace(-1, 1, 32)).cuda())


def test_not_finite_and_zeros():
    x = torch.ones(4, 96, device="cuda")
    x[0, 5], x[1, 40], x[2, 95] = float("inf"), float("nan"), -float("inf")
    x[3] = 0
    x[3, 1] = -0.0
    for t in DT.values():
        codes, scales = _same(x.to(t))
        out = torch.empty(4, 96, dtype=t, device="cuda")
        q.moe_act8_load(codes, scales, out, q.make_grouped_workspace())
        bad = ~torch.isfinite(x).reshape(4, 3, 32).all(dim=2).repeat_interleave(32, dim=1)
        assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], x.to(t)[~bad])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens,cols,top_k,spare", [(1, 32, 1, 0), (1, 2048, 8, 0), (37, 160, 3, 5), (300, 2080, 8, 0)])
def test_load_into_slots(tokens, cols, top_k, spare, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, cols, generator=g, device="cuda").to(DT[dtype])
    codes, scales = _save(x)
    perm = torch.randperm(tokens * top_k, generator=g, device="cuda").int()
    out = torch.full((tokens * top_k + spare, cols), 7.0, dtype=DT[dtype], device="cuda")
    ws = q.make_grouped_workspace()
    q.moe_act8_load(codes, scales, out, ws, perm=perm, top_k=top_k)
    vals = torch.from_numpy(step.act8_load(codes.cpu().numpy(), scales.cpu().numpy())).cuda()
    n = perm.numel()
    assert torch.equal(out[:n], vals[(perm // top_k).long()].to(DT[dtype])) and (out[n:] == 7).all()
    straight = torch.empty_like(x)
    q.moe_act8_load(codes, scales, straight, ws)
    assert torch.equal(straight, vals.to(DT[dtype]))
    assert q.moe_get_device_status(ws) == q.STRATA_OK


def test_load_every_code_and_scale():
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, device="cuda", dtype=torch.uint8)[:, None].repeat(1, 8)
    want = torch.from_numpy(step.act8_load(codes.cpu().numpy(), np.minimum(scales.cpu().numpy(), 254))).cuda()
    nan = torch.isnan(want)
    for name, t in DT.items():
        out = torch.empty(256, 256, dtype=t, device="cuda")
        q.moe_act8_load(codes, scales, out, q.make_grouped_workspace())
        ref = want.clamp(-65504, 65504).half() if name == "fp16" else want.float().to(t)
        rows = slice(1, 248)                    # the scales that finite blocks get
        assert torch.equal(torch.isnan(out)[rows], nan[rows])
        assert torch.equal(out[rows][~nan[rows]], ref[rows][~nan[rows]])
        assert (out[0][~nan[0]] == 0).all()


def test_bad_source_rows_read_as_zeros():
    x = torch.ones(4, 64, device="cuda", dtype=torch.bfloat16)
    codes, scales = _save(x)
    perm = torch.tensor([0, 7, 8, -1, 3, -2 ** 31], dtype=torch.int32, device="cuda")
    out, ws = torch.full((6, 64), 7.0, dtype=torch.bfloat16, device="cuda"), q.make_grouped_workspace()
    q.moe_act8_load(codes, scales, out, ws, perm=perm, top_k=2)
    assert out[:, 0].tolist() == [1, 1, 0, 0, 1, 0] and (out == out[:, :1]).all()
    assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
