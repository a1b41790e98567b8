"""The grouped products' and the 4-bit formats' argument checks (no GPU: all
of them come before any CUDA call), sizes, and the plain forms' own pins."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from quantized_moe_expert_fwd_gb300 import build as qbuild
from tests import grouped_ref as ref

P = 1 << 20          # an aligned address that no refused call reads
WS = 65536


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load()


def _mm(lib, fn="moe_grouped_mm", dtype=0, a=P, b=P, M=4, K=64, N=64, E=2, off=P, od=0, out=P, ws=P,
        n=WS):
    return getattr(lib, fn)(dtype, a, b, M, K, N, E, off, od, out, ws, n, None)


BAD_MM = [dict(dtype=2), dict(dtype=-1), dict(od=1), dict(od=3), dict(M=-1), dict(K=0), dict(N=0),
          dict(K=(1 << 20) + 1), dict(N=(1 << 20) + 1), dict(E=0), dict(E=1025), dict(a=0),
          dict(b=0), dict(out=0), dict(off=0), dict(a=P + 8), dict(b=P + 2), dict(out=P + 4),
          dict(off=P + 2), dict(ws=0), dict(ws=P + 16), dict(n=WS - 1)]


@pytest.mark.parametrize("fn", ["moe_grouped_mm", "moe_grouped_mm_dx", "moe_grouped_mm_dw"])
@pytest.mark.parametrize("kw", BAD_MM, ids=str)
def test_grouped_mm_refusals(lib, fn, kw):
    assert _mm(lib, fn, **kw) == q.STRATA_EINVAL


def test_no_rows_launch_nothing(lib):
    for fn in ("moe_grouped_mm", "moe_grouped_mm_dx"):
        assert _mm(lib, fn, M=0, a=0, out=0) == q.STRATA_OK
    assert lib.moe_fp4_quantize(0, 0, None, 0, 64, None, 1, 0, P, 2, 0, None, None, 0, None, 0,
                                None) == q.STRATA_OK
    assert lib.moe_fp4_dequantize(1, None, None, 0, 0, 64, P, 2, 0, 0, None, None, 0,
                                  None) == q.STRATA_OK
    assert lib.moe_grouped_mm_fp4(1, None, None, 0, P, P, 1 << 30, 0, 64, 64, 2, P, None, 0, 0, None,
                                  None, 0, None) == q.STRATA_OK


def test_workspace_and_scale_bytes(lib):
    assert q.moe_grouped_workspace_bytes() == WS
    # 128 rows by 4 scales a tile: 64 columns a word in NV, 128 in MX
    assert q.moe_fp4_scale_bytes(q.FP4_NV, 128, 64) == 512
    assert q.moe_fp4_scale_bytes(q.FP4_MX, 128, 64) == 512
    assert q.moe_fp4_scale_bytes(q.FP4_NV, 129, 96) == 2 * 2 * 512
    assert q.moe_fp4_scale_bytes(q.FP4_MX, 256 * 1024, 2048, 256) == 256 * 8 * 16 * 512
    # ragged: a block of its own for every group that can have rows
    assert q.moe_fp4_scale_bytes(q.FP4_NV, 300, 64, 7, ragged=True) == (2 + 7) * 512
    assert q.moe_fp4_scale_bytes(q.FP4_NV, 3, 64, 7, ragged=True) == 3 * 512
    for bad in ((2, 8, 64, 1), (0, -1, 64, 1), (0, 8, 48, 1), (0, 8, 16, 1), (0, 8, 64, 0),
                (0, 8, 64, 3), (0, 2048, 64, 1025)):
        assert q.moe_fp4_scale_bytes(*bad) == 0, bad
    # the worst offsets need no more than the ragged size: every split of small row counts
    for counts in ([1, 1, 1], [129, 1], [128, 128, 1], [0, 257, 0], [5], [127, 2, 127]):
        _, used = ref.tile_places(counts, 64, 1)
        assert used <= q.moe_fp4_scale_bytes(q.FP4_NV, sum(counts), 64, len(counts), ragged=True)


def _quant(lib, fmt=0, dtype=0, x=P, x_rows=4, cols=64, perm=0, top_k=1, rows=4, off=P, groups=2,
           ex=0, codes=P, sc=P, scn=1 << 20, ws=P, n=WS):
    return lib.moe_fp4_quantize(fmt, dtype, x, x_rows, cols, perm, top_k, rows, off, groups, ex,
                                codes, sc, scn, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(fmt=2), dict(fmt=-1), dict(dtype=3), dict(x=0), dict(x=P + 8), dict(x_rows=-1), dict(x_rows=3),
    dict(cols=0), dict(cols=48), dict(cols=(1 << 20) + 32), dict(perm=P + 2), dict(top_k=0),
    dict(rows=-1, x_rows=-1), dict(off=P + 1), dict(off=0, groups=3), dict(groups=0),
    dict(groups=1025), dict(ex=1), dict(fmt=1, ex=65), dict(fmt=1, ex=-65), dict(codes=0),
    dict(codes=P + 8), dict(sc=0), dict(sc=P + 8), dict(scn=1023), dict(ws=0), dict(n=100)], ids=str)
def test_quantize_refusals(lib, kw):
    assert _quant(lib, **kw) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", [
    dict(fmt=2), dict(codes=0), dict(sc=0), dict(scn=1023), dict(rows=-1), dict(cols=33),
    dict(off=P + 2), dict(groups=0), dict(ex=3), dict(od=3), dict(od=-1), dict(out=0),
    dict(out=P + 4), dict(ws=P + 128), dict(n=0)], ids=str)
def test_dequantize_refusals(lib, kw):
    a = dict(fmt=0, codes=P, sc=P, scn=1 << 20, rows=4, cols=64, off=P, groups=2, ex=0, od=0, out=P,
             ws=P, n=WS) | kw
    assert lib.moe_fp4_dequantize(a["fmt"], a["codes"], a["sc"], a["scn"], a["rows"], a["cols"],
                                  a["off"], a["groups"], a["ex"], a["od"], a["out"], a["ws"], a["n"],
                                  None) == q.STRATA_EINVAL


@pytest.mark.parametrize("kw", [
    dict(fmt=2), dict(xq=0), dict(xs=P + 4), dict(xsn=1023), dict(wq=P + 8), dict(wsc=0),
    dict(wscn=1023), dict(M=-1), dict(K=16), dict(K=0), dict(N=0), dict(N=65, swiglu=1), dict(E=0),
    dict(off=0), dict(alpha=P + 1), dict(od=3), dict(y=0), dict(ws=0), dict(n=8)], ids=str)
def test_grouped_mm_fp4_refusals(lib, kw):
    a = dict(fmt=0, xq=P, xs=P, xsn=1 << 20, wq=P, wsc=P, wscn=1 << 20, M=4, K=64, N=64, E=2, off=P,
             alpha=0, swiglu=0, od=0, y=P, ws=P, n=WS) | kw
    assert lib.moe_grouped_mm_fp4(a["fmt"], a["xq"], a["xs"], a["xsn"], a["wq"], a["wsc"], a["wscn"],
                                  a["M"], a["K"], a["N"], a["E"], a["off"], a["alpha"], a["swiglu"],
                                  a["od"], a["y"], a["ws"], a["n"], None) == q.STRATA_EINVAL


def test_binding_takes_cuda_tensors_only(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(WS, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        q.moe_grouped_mm(x, w, off, torch.zeros(4, 64, dtype=torch.bfloat16), ws)
    with pytest.raises(ValueError, match="shape"):
        q.moe_grouped_mm(x, w, off, torch.zeros(5, 64, dtype=torch.bfloat16), ws)
    with pytest.raises(ValueError, match="CUDA"):
        q.moe_fp4_quantize(x, x, x, q.FP4_MX, ws)


# --------------------------------------------------------- the plain forms
def test_plain_quantize_hand_computed():
    # MX: amax 6 -> 2^(2 - 2): values keep, ties go to the even code, 5 -> 4, beyond 6 saturates
    x = np.zeros((1, 32))
    x[0, :10] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.3]
    c, s = ref.quantize(x, 0)
    assert s[0, 0] == 127
    assert list(c[0, :10]) == [7, 15, 0, 2, 2, 4, 4, 6, 6, 9]
    x[0, 0] = 7.9
    c, s = ref.quantize(x, 0)
    assert s[0, 0] == 127 and c[0, 0] == 7
    x[0, 0] = 8.0
    assert ref.quantize(x, 0)[1][0, 0] == 128
    # NV: amax 6 -> scale 1 = 0x38; amax 6 * 448 -> 0x7e; below half of 2^-9 -> 0
    y = np.zeros((1, 16))
    # (the last: 1.5 smallest steps round to 2, and 9 / 2 = 4.5 is nearer 4, code 6)
    for amax, byte, code in ((6.0, 0x38, 15), (6 * 448.0, 0x7e, 15), (1e9, 0x7e, 15),
                             (6 * 2.0 ** -9, 1, 15), (6 * 2.0 ** -10, 0, 0),
                             (6 * 1.5 * 2.0 ** -9, 2, 14)):
        y[0, 3] = -amax
        c, s = ref.quantize(y, 1)
        assert s[0, 0] == byte and c[0, 3] == code, amax
    y[0, 0] = np.nan
    assert ref.quantize(y, 1)[1][0, 0] == 0x7f
    # every code and scale reads back
    for fmt in (0, 1):
        codes = np.tile(np.arange(16, dtype=np.uint8), (1, 4))
        s = np.full((1, 64 // ref.VEC[fmt]), 0x38 if fmt else 127, dtype=np.uint8)
        v = ref.values(codes, s, fmt)
        assert np.array_equal(v[0, :8], ref.GRID) and np.array_equal(v[0, 8:16], -ref.GRID)
        assert np.array_equal(ref.quantize(v, fmt)[0] & 7, codes & 7)


def test_plain_tiles_hand_computed():
    place, used = ref.tile_places([1, 130], 128, 1)          # 2 words a row
    assert used == 3 * 2 * 512
    assert list(place[0]) == [0, 1, 2, 3, 512, 513, 514, 515]
    assert place[1][0] == 1024 and place[2][0] == 1024 + 16 and place[33][0] == 1024 + 4
    assert place[1 + 128][0] == 2048 and place[1 + 129][7] == 2048 + 512 + 16 + 3
