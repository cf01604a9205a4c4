"""nvfp4 with dropout: the matrix scale that the kept values need."""
import numpy as np
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests import fp4_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_the_largest_kept_values_are_held(rounding):
    """Equal magnitudes are the largest of every block: with the scale of the kept values they are held to
    FP32's rounding of scale and product, and with x's own they come out as x itself."""
    x = torch.full((64, 256), 3.0, device=DEV)
    x[:, ::3] = -3.0
    p, kept = 0.25, 49152
    keep = ref.bits16(64, 256, 8, 0, 0) < kept
    for larger, want in ((65536 / kept, 4.0), (1.0, 3.0)):
        g = torch.tensor([3.0 * larger / 2688], device=DEV)
        for q in (ptc.quantize_fp4(x, "nvfp4", rounding=rounding, tensor_scale=g, p=p, seed=8),
                  ptc.quantize_fp4(x, "nvfp4", transposed="both", rounding=rounding, tensor_scale=g, p=p, seed=8)[0]):
            v = ptc.dequantize_fp4(q, torch.float32).cpu().double().numpy()
            assert np.all(v[~keep] == 0)
            assert np.all(np.abs(np.abs(v[keep]) - want) <= want * 2.0 ** -22)
