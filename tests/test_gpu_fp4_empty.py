"""Matrices of no rows and of no values: their scales by rows."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,K", [(0, 0), (0, 40), (5, 0), (200, 0)])
def test_row_scales(rows, K, fmt):
    import __graft_entry__
    __graft_entry__.build()
    for q in (ptc.quantize_fp4(torch.zeros(rows, K, device=DEV), fmt),
              ptc.quantize_fp4(torch.zeros(K, rows, device=DEV), fmt, transposed=True)):
        s = q.row_scales()
        assert s.shape == (rows, -(-K // (32 if fmt == "mxfp4" else 16))) and s.dtype == torch.uint8
        assert ptc.Fp4Matrix.tile_scales(s).numel() == q.scales.numel() == ptc.fp4_scale_bytes(rows, K, fmt)
