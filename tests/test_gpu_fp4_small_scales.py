"""nvfp4 quantisation with matrix scales from zero up to the smallest normal numbers and beyond.

Codes and scale bytes are functions of the inputs to the last bit and are
compared for equality; with a matrix scale of zero both are zero."""
import numpy as np
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests import fp4_ref as ref
from tests.gpu_util import DEV
from tests.test_gpu_fp4 import check_quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def both_ways(x, g, rounding, p=0.0):
    """Rows alone, columns alone, and both in one pass against the reference."""
    xn = x.cpu().float().numpy()
    rows, cols = xn.shape
    bits = ref.bits16(rows, cols, 3, 1, 1) if rounding == "stochastic" else None
    tb = None if bits is None else bits.T
    t = torch.tensor([g], dtype=torch.float32, device=DEV)
    assert t.item() == g
    kw = dict(rounding=rounding, tensor_scale=t, seed=3, offset=1)
    xt = np.ascontiguousarray(xn.T)
    check_quantised(ptc.quantize_fp4(x, "nvfp4", **kw), xn, "nvfp4", rounding, bits, np.float32(g))
    check_quantised(ptc.quantize_fp4(x, "nvfp4", transposed=True, **kw), xt, "nvfp4", rounding, tb, np.float32(g))
    a, b = ptc.quantize_fp4(x, "nvfp4", transposed="both", **kw)
    check_quantised(a, xn, "nvfp4", rounding, bits, np.float32(g))
    check_quantised(b, xt, "nvfp4", rounding, tb, np.float32(g))


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [-149, -147, -140, -133, -128, -126, -125, -118, -110, -104, -60, -51, -50, -49, 100])
def test_matrix_scale_of_every_size(e, dtype, rounding):
    rng = np.random.default_rng(e + 200)
    x = rng.standard_normal((72, 144)) * np.exp2(rng.integers(-12, 13, (72, 144))) * 2.0 ** min(e + 11, 112)
    x[rng.random(x.shape) < 0.2] = 0.0
    x[5] = 0.0
    x[7, 16:32] = 3e38
    x[9, ::3] = 2.0 ** -126
    x[11, ::5] = -1e-45
    with np.errstate(over="ignore"):
        x = torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)
    both_ways(x, float(np.float32(2.0 ** e)), rounding)


def test_largest_magnitude_as_the_scale_of_tiny_values():
    """The usual choice, largest magnitude / 2688, for values so small that it is a subnormal number."""
    for size in (1e-36, 1e-38, 1e-41):
        x = (torch.randn(64, 96, generator=torch.Generator().manual_seed(1)) * size).to(DEV)
        x[:, ::7] = 0.0
        both_ways(x, (x.abs().amax() / 2688).item(), "nearest")
        both_ways(x, (x.abs().amax() / 2688).item(), "stochastic")


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("value", [0.0, 1.0, -3e38])
def test_a_matrix_scale_of_zero_gives_zeros(value, rounding):
    x = torch.full((40, 80), value, device=DEV)
    x[3, 5] = 0.0
    zero = torch.zeros(1, device=DEV)
    one = ptc.quantize_fp4(x, "nvfp4", rounding=rounding, tensor_scale=zero)
    for q in (one, *ptc.quantize_fp4(x, "nvfp4", transposed="both", rounding=rounding, tensor_scale=zero)):
        assert not (ref.unpack(q.codes.cpu().numpy()) & 7).any() and not q.scales.any()
        assert not ptc.dequantize_fp4(q).any() and not ptc.matmul_fp4(q, q).any()
    x[3, 5] = float("nan")
    q = ptc.quantize_fp4(x, "nvfp4", rounding=rounding, tensor_scale=zero)
    s = q.row_scales().cpu().numpy()
    assert s[3, 0] == 0x7F and np.count_nonzero(s) == 1
