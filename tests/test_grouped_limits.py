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
