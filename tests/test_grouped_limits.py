"""Sizes past what the grouped calls count in 32 bits are refused, not wrapped
(no GPU: the refusals come before any CUDA call)."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from quantized_moe_expert_fwd_gb300 import build as qbuild

P = 1 << 20          # an aligned address that no refused call reads
WS = 65536
MOST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load()


@pytest.mark.parametrize("rows", [MOST + 1, 2 ** 31 - 256, 2 ** 31 - 128, 2 ** 31 - 1])
def test_rows_that_a_block_count_would_overflow(lib, rows):
    """A group of 2^31 - 256 rows and more plus a tile's height passes 2^31: it would count as no tiles."""
    for fn in ("moe_grouped_mm", "moe_grouped_mm_dx", "moe_grouped_mm_dw"):
        assert getattr(lib, fn)(0, P, P, rows, 8, 8, 1, P, 0, P, P, WS, None) == q.STRATA_EINVAL
    n = 1 << 50
    assert lib.moe_fp4_quantize(0, 0, P, rows, 32, None, 1, rows, P, 1, 0, P, P, n, P, WS,
                                None) == q.STRATA_EINVAL
    assert lib.moe_fp4_dequantize(0, P, P, n, rows, 32, P, 1, 0, 0, P, P, WS, None) == q.STRATA_EINVAL
    assert lib.moe_grouped_mm_fp4(0, P, P, n, P, P, n, rows, 32, 8, 1, P, None, 0, 0, P, P, WS,
                                  None) == q.STRATA_EINVAL
    assert q.moe_fp4_scale_bytes(q.FP4_MX, rows, 32) == 0
    assert q.moe_fp4_scale_bytes(q.FP4_MX, rows, 32, ragged=True) == 0


def test_most_rows_have_scale_bytes(lib):
    assert q.moe_fp4_scale_bytes(q.FP4_MX, MOST, 32) == MOST // 128 * 512
    assert q.moe_fp4_scale_bytes(q.FP4_NV, MOST, 32, 7, ragged=True) == (MOST // 128 + 7) * 512


BIG = 2 ** 32 + 8    # passed on in 32 bits it would read as 8


def _meta(*shape, dtype=torch.bfloat16):
    """A tensor of that shape without memory."""
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("M,K,N", [(BIG, 8, 8), (8, BIG, 8), (8, 8, BIG)])
def test_binding_refuses_products_past_32_bits(lib, M, K, N):
    x, w, dy = _meta(M, K), _meta(1, N, K), _meta(M, N)
    off, ws = _meta(2, dtype=torch.int32), _meta(WS, dtype=torch.uint8)
    for call in (lambda: q.moe_grouped_mm(x, w, off, dy, ws), lambda: q.moe_grouped_mm_dx(dy, w, off, x, ws),
                 lambda: q.moe_grouped_mm_dw(dy, x, off, w, ws)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_binding_refuses_4bit_sizes_past_32_bits(lib):
    u8 = torch.uint8
    ws, off, sc = _meta(WS, dtype=u8), _meta(2, dtype=torch.int32), _meta(512, dtype=u8)
    x, codes, out = _meta(8, 32), _meta(8, 16, dtype=u8), _meta(8, 32)
    long_x, long_codes = _meta(BIG, 32), _meta(BIG, 16, dtype=u8)
    wq, y = _meta(1, 8, 16, dtype=u8), _meta(8, 8)
    perm = _meta(8, dtype=torch.int32)
    for call in (lambda: q.moe_fp4_quantize(long_x, codes, sc, 0, ws, perm=perm),
                 lambda: q.moe_fp4_quantize(x, long_codes, sc, 0, ws),
                 lambda: q.moe_fp4_quantize(x, codes, sc, BIG, ws),
                 lambda: q.moe_fp4_quantize(x, codes, sc, 0, ws, n_groups=BIG),
                 lambda: q.moe_fp4_quantize(x, codes, sc, 1, ws, scale_exp=-BIG),
                 lambda: q.moe_fp4_quantize(x, codes, sc, 0, ws, perm=perm, top_k=BIG),
                 lambda: q.moe_fp4_dequantize(long_codes, sc, _meta(BIG, 32), 0, ws),
                 lambda: q.moe_fp4_dequantize(codes, sc, out, 0, ws, scale_exp=BIG),
                 lambda: q.moe_fp4_dequantize(codes, sc, out, 2 ** 32, ws),
                 lambda: q.moe_fp4_dequantize(codes, sc, out, 0, ws, n_groups=BIG),
                 lambda: q.moe_grouped_mm_fp4(long_codes, sc, wq, sc, off, _meta(BIG, 8), 0, ws),
                 lambda: q.moe_grouped_mm_fp4(codes, sc, _meta(1, BIG, 16, dtype=u8), sc, off,
                                              _meta(8, BIG), 0, ws),
                 lambda: q.moe_grouped_mm_fp4(codes, sc, wq, sc, off, y, 2 ** 32 + 1, ws)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_binding_scale_bytes_past_32_bits(lib):
    for bad in ((0, BIG, 64, 1), (0, 128, 2 ** 32 + 64, 1), (2 ** 32, 128, 64, 1), (0, 128, 64, 2 ** 32 + 1)):
        assert q.moe_fp4_scale_bytes(*bad) == 0, bad
