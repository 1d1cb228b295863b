"""Register budgets of the 8-bit and balance kernels, from the compiler's
resource report: none of them spills, and those whose speed rests on several
wavefronts per SIMD keep them. CPU only (compiles, runs nothing)."""
from __future__ import annotations

import shutil

import pytest

from tests.test_kernel_resources import HIPCC, _report

pytestmark = pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not installed")


def test_products_do_not_spill():
    """The 256 x 256 tile stands at 249 of 256 VGPRs, 128 x 256 with fp32 sums
    at 194; the streaming kernel keeps two workgroups of eight wavefronts per CU."""
    rep = _report("gemm_fp8.hip")
    stream = {k: v for k, v in rep.items() if "fp8_stream_kernel" in k}
    tiles = {k: v for k, v in rep.items() if "fp8_tile_kernel" in k}
    # K split over 1, 2, 4 and 8 wavefronts, two out types; ten tiles in three forms, the largest in one
    # (32 x 64 has stages of its own for fp32 sums)
    assert len(stream) == 8 and len(tiles) == 31 and len(rep) == 39, list(rep)
    for name, v in rep.items():
        assert v["scratch"] == 0 and v["waves"] >= 2, (name, v)
    for name, v in stream.items():
        assert v["waves"] >= 4, (name, v)


@pytest.mark.parametrize("src,kernels", [("quant_fp8.hip", 8), ("balance.hip", 11)])
def test_rows_and_balance_do_not_spill(src, kernels):
    """Bound by memory or latency: at least half of the SIMD's eight wavefronts."""
    rep = _report(src)
    assert len(rep) == kernels, list(rep)
    for name, v in rep.items():
        assert v["scratch"] == 0 and v["waves"] >= 5, (name, v)
