"""The linear layer's input gradient is rounded once.

Operands that mxfp4 holds exactly make the product an integer, exact in FP32, so
dx is one FP32 product with dropout's scale and one rounding to dy's type: it is
compared for equality."""
import numpy as np
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from precision_tensor_core_gb300 import fp4_linear
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


def held(rng, rows, cols):
    """Integers that mxfp4 holds exactly along the rows and along the columns."""
    v = rng.choice(np.array([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], dtype=np.float32), size=(rows, cols))
    v[:, ::32] = 6.0
    v[::32, :] = 6.0
    return v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,inputs,outputs,p", [(1, 32, 32, 0.25), (65, 203, 96, 0.1), (128, 256, 512, 0.3)])
def test_dx_is_rounded_once(tokens, inputs, outputs, p, dtype):
    rng = np.random.default_rng(tokens)
    dy, w = held(rng, tokens, outputs), held(rng, outputs, inputs)
    x = torch.ones(tokens, inputs, dtype=dtype, device=DEV)
    _, saved = fp4_linear.forward(x, torch.from_numpy(w).to(DEV, dtype), p=p, seed=11, offset=3)
    dx, _ = fp4_linear.backward(torch.from_numpy(dy).to(DEV, dtype), saved)
    product = dy.astype(np.float64) @ w.astype(np.float64)
    assert np.abs(product).max() < 2 ** 24  # exact in FP32
    want = torch.from_numpy(ref.dropout(product.astype(np.float32), p, 11, 3)).to(dtype)
    assert dx.dtype == dtype and torch.equal(dx.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (33, 1000), (130, 257), (9, 4100)])
def test_float32_dropped_out_to_16_bits(rows, cols, dtype):
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(cols)).to(DEV)
    want = torch.from_numpy(ref.dropout(x.cpu().numpy(), 0.3, 7, 1 << 40)).to(dtype)
    y = ptc.dropout(x, 0.3, 7, 1 << 40, out_dtype=dtype)
    assert y.dtype == dtype and torch.equal(y.cpu(), want)
    wide = torch.full((rows, cols + 3), 5.0, dtype=dtype, device=DEV)
    assert torch.equal(ptc.dropout(x, 0.3, 7, 1 << 40, out=wide[:, 1:cols + 1], out_dtype=dtype).cpu(), want)
    assert torch.all(wide[:, 0] == 5) and torch.all(wide[:, cols + 1:] == 5)


def test_out_dtype_refusals():
    x = torch.zeros(4, 64, device=DEV)
    h = x.bfloat16()
    for bad in (lambda: ptc.dropout(x, 0.1, 1, out=h), lambda: ptc.dropout(x, 0.1, 1, out=x, out_dtype=h.dtype),
                lambda: ptc.dropout(x, 0.1, 1, residual=x, out_dtype=h.dtype)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ptc.dropout(x, 0.1, 1, residual=h, out_dtype=h.dtype),
                lambda: ptc.dropout(h, 0.1, 1, out_dtype=torch.float32),
                lambda: ptc.dropout(h, 0.1, 1, out_dtype=torch.float16),
                lambda: ptc.dropout(x, 0.1, 1, out=x.view(torch.bfloat16)[:, :64], out_dtype=h.dtype)):
        with pytest.raises(ptc.PtcError):
            bad()
    for bad in (lambda: ptc.dropout(x, 0.1, 1, out_dtype=torch.float64), lambda: ptc.dropout(x, 0.1, 1, out_dtype="f16")):
        with pytest.raises(TypeError):
            bad()
