"""Long reductions of one sign in the grouped products.

The tensor cores truncate as they add.  With terms of one sign the losses do
not cancel: they grow with the number of additions.  So the accumulator is
drained after a number of terms that depends on the output's type, and the
pieces are added in fp32 with rounding.

The limit, relative to the sum S of `terms` positive terms: a piece takes a
truncated addition for 16 terms, which loses at most two steps (2^-23) of the
partial sum.  A piece's partial sums are half of it on average, so all the
pieces together lose at most (terms of a piece / 16) 2^-23 S; joining them takes one rounded addition a
piece, and 8 more where a cluster splits the reduction, each off by at most
2^-24 S.  Then the output's own rounding.  Without drains `terms` takes the
piece's place."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import grouped_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PIECE = {"bf16": 2048, "fp16": 2048, "fp32": 512}
PIECE_FP4 = {"bf16": 8192, "fp16": 8192, "fp32": 2048}
TYPES = [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp16")]


def _sum_limit(terms, piece):
    return min(terms, piece) / 16 * 2.0 ** -23 + (-(-terms // piece) + 8) * 2.0 ** -24


def _check(got, want, limit):
    """Elementwise, and on average: the output's roundings (uniform within half a step, so
    eps / 2 / sqrt(3) their deviation at most) cancel over the values, truncation does not."""
    rel = (got.double() - want) / want
    half = torch.finfo(got.dtype).eps / 2
    worst, mean = float(rel.abs().max()), float(rel.mean())
    print(f"worst {worst:.2e} (limit {limit + half * (1 + limit):.2e}), mean {mean:.2e} (limit {limit:.2e})")
    assert worst <= limit + half * (1 + limit)
    assert abs(mean) <= limit + 5 * half / 3 ** 0.5 / rel.numel() ** 0.5


def _positive(g, dtype, scale, *shape):
    return ((1 + torch.rand(*shape, generator=g, device="cuda")) * scale).to(DT[dtype])


# direction, rows of each group, K, N and the kernel that the sizes pick: the reduction split over a
# cluster, one CTA a tile of 128 or of 256 columns, a pair of CTAs
CASES = {
    "forward_split": ("forward", [40], 1 << 18, 136),
    "forward_columns": ("forward", [9] * 60, 1 << 16, 264),
    "forward_single": ("forward", [100] * 40, 1 << 15, 1024),
    "forward_pair": ("forward", [2048], 1 << 15, 2048),
    "dx_split": ("dx", [40], 136, 1 << 18),
    "dx_single": ("dx", [100] * 40, 1024, 1 << 15),
    "dx_pair": ("dx", [2048], 2048, 1 << 15),
    "dw_single": ("dw", [1 << 18] + [0] * 599, 64, 72),
    "dw_pair": ("dw", [(1 << 18) - 7], 264, 136),
}


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("name", CASES)
def test_products(name, dtype, out):
    way, counts, K, N = CASES[name]
    M, E = sum(counts), len(counts)
    terms = {"forward": K, "dx": N, "dw": counts[0]}[way]
    g = torch.Generator(device="cuda").manual_seed(len(name))
    s = terms ** -0.5                                   # sums between 1 and 4
    off, ws = ref.offsets_of(counts).cuda(), q.make_grouped_workspace()
    a = _positive(g, dtype, s, M, N if way == "dx" else K)
    if way == "dw":
        b = _positive(g, dtype, s, M, N)
        got = torch.zeros(E, N, K, dtype=DT[out], device="cuda")
        q.moe_grouped_mm_dw(b, a, off, got, ws)
        got, want = got[0], b.double().T @ a.double()
    else:
        b = _positive(g, dtype, s, E, N, K)
        got = torch.zeros(M, K if way == "dx" else N, dtype=DT[out], device="cuda")
        (q.moe_grouped_mm_dx if way == "dx" else q.moe_grouped_mm)(a, b, off, got, ws)
        want = torch.empty(got.shape, dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(ref.spans(off)):
            we = b[e].double()
            want[lo:hi] = a[lo:hi].double() @ (we if way == "dx" else we.T)
    _check(got, want, _sum_limit(terms, PIECE[out]))
    assert q.moe_get_device_status(ws) == q.STRATA_OK


# direction, rows, K, N, terms of a piece of the sum: the kernels on the CUDA cores (few rows, few
# columns, widths of any kind), and two on the tensor cores
EQUAL = {
    "few_rows": ("forward", 5, 1 << 20, 40, 256),
    "few_columns": ("forward", 700, 1 << 18, 3, 256),
    "any_width": ("forward", 70, (1 << 17) + 3, 51, 512),
    "any_width_dx": ("dx", 70, 51, (1 << 17) + 3, 512),
    "any_width_dw": ("dw", (1 << 18) - 7, 37, 51, 512),
    "tensor_cores": ("forward", 40, 1 << 18, 136, None),
    "tensor_cores_dw": ("dw", (1 << 18) - 7, 264, 136, None),
}


@pytest.mark.parametrize("value", [1.1, 1.3])
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("name", EQUAL)
def test_equal_terms(name, dtype, out, value):
    """Equal terms round the same way within a binade.  On the CUDA cores an addition is off by at most
    2^-24 of its partial sum, and n partial sums add up to (n + 1) / 2 whole ones: (p + 1) / 2 for the
    p terms of a piece, (c + 1) / 2 for a lane's c pieces, 6 for the lanes' sum."""
    way, M, K, N, piece = EQUAL[name]
    terms = {"forward": K, "dx": N, "dw": M}[way]
    off, ws = ref.offsets_of([M]).cuda(), q.make_grouped_workspace()
    v = torch.tensor(value * terms ** -0.5, device="cuda").to(DT[dtype])

    def same(*shape):
        return v.expand(*shape).contiguous()
    if way == "dw":
        got = torch.zeros(1, N, K, dtype=DT[out], device="cuda")
        q.moe_grouped_mm_dw(same(M, N), same(M, K), off, got, ws)
    else:
        got = torch.zeros(M, K if way == "dx" else N, dtype=DT[out], device="cuda")
        call = q.moe_grouped_mm_dx if way == "dx" else q.moe_grouped_mm
        call(same(M, N if way == "dx" else K), same(1, N, K), off, got, ws)
    want = float(v.double()) ** 2 * terms
    if piece is None:
        limit = _sum_limit(terms, PIECE[out])
    else:
        lanes = 32 if piece == 256 else 1
        limit = ((piece + 1) / 2 + (terms / lanes / piece + 2) / 2 + 6) * 2.0 ** -24
    half = torch.finfo(DT[out]).eps / 2
    worst = float(((got.double() - want) / want).abs().max())
    assert worst <= limit + half * (1 + limit), f"{worst:.2e}"
    assert q.moe_get_device_status(ws) == q.STRATA_OK


def _places(rows, n, words):
    """The byte of each scale of one group's rows."""
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(n, device="cuda")[None]
    return (r // 128 * words + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4


def _fp4(g, fmt, rows, K, nbytes):
    """Positive codes (1 to 6) and scales near one: (packed, tiled scales, float64 values)."""
    vec = ref.VEC[fmt]
    codes = torch.randint(2, 8, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
    lo, hi = (126, 129) if fmt == 0 else (0x30, 0x40)
    sb = torch.randint(lo, hi, (rows, K // vec), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == 0:
        s = torch.exp2(sb.double() - 127)
    else:
        s = (8 + (sb & 7)).double() * torch.exp2((sb >> 3).double() - 10)
    tiles = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    tiles[_places(rows, K // vec, -(-K // (4 * vec)))] = sb
    v = torch.from_numpy(ref.GRID).cuda()[codes.long()] * s.repeat_interleave(vec, dim=1)
    return codes[:, 0::2] | codes[:, 1::2] << 4, tiles, v


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("fmt", [pytest.param(0, id="mx"), pytest.param(1, id="nv")])
def test_4bit_product(fmt, out):
    M, K, N = 33, 1 << 20, 72
    g = torch.Generator(device="cuda").manual_seed(fmt)
    xq, xs, xv = _fp4(g, fmt, M, K, q.moe_fp4_scale_bytes(fmt, M, K, 1, True))
    wq, wsc, wv = _fp4(g, fmt, N, K, q.moe_fp4_scale_bytes(fmt, N, K, 1))
    off, ws = ref.offsets_of([M]).cuda(), q.make_grouped_workspace()
    y = torch.zeros(M, N, dtype=DT[out], device="cuda")
    alpha = torch.full((1,), 2.0 ** -20, device="cuda")
    q.moe_grouped_mm_fp4(xq, xs, wq[None], wsc, off, y, fmt, ws, alpha=alpha)
    _check(y, xv @ wv.T * 2.0 ** -20, _sum_limit(K, PIECE_FP4[out]))
    assert q.moe_get_device_status(ws) == q.STRATA_OK
