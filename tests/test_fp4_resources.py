"""Register budgets of the 4-bit, sort and row kernels, from the compiler's
resource report: none of them spills, and those bound by memory keep several
wavefronts per SIMD. CPU only (compiles, runs nothing)."""
from __future__ import annotations

import shutil

import pytest

from tests.test_kernel_resources import HIPCC, _report

pytestmark = pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not installed")


def test_products_do_not_spill():
    """The 256 x 256 tile stands at all 256 VGPRs of two wavefronts per SIMD; the
    streaming kernel keeps two workgroups of eight wavefronts per CU."""
    rep = _report("gemm_fp4.hip")
    stream = {k: v for k, v in rep.items() if "fp4_stream_kernel" in k}
    tiles = {k: v for k, v in rep.items() if "fp4_tile_kernel" in k}
    # K split over 2, 4 and 8 wavefronts, two out types, two ways to load scales; seven tiles with scales by
    # 16 and 4 bytes, weights read once or not, and by single bytes; the largest by 16 bytes only
    assert len(stream) == 12 and len(tiles) == 7 * 5 + 2 and len(rep) == 49, list(rep)
    for name, v in rep.items():
        assert v["scratch"] == 0 and v["waves"] >= 2, (name, v)
    for name, v in stream.items():
        assert v["waves"] >= 4, (name, v)


@pytest.mark.parametrize("src,kernels,waves", [("quant_fp4.hip", 12, 5), ("routes.hip", 33, 3)])
def test_rows_and_sort_do_not_spill(src, kernels, waves):
    rep = _report(src)
    assert len(rep) == kernels, list(rep)
    for name, v in rep.items():
        assert v["scratch"] == 0 and v["waves"] >= waves, (name, v)
