"""The 4-bit operators and autograd: no gradient is lost without an error, and writes in place are seen."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from precision_tensor_core_gb300 import fp4_linear
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def test_tensors_that_require_grad_are_refused():
    x = torch.randn(4, 64, device=DEV).bfloat16().requires_grad_()
    y = torch.randn(4, 64, device=DEV).bfloat16()
    w = ptc.quantize_fp4(torch.randn(32, 64, device=DEV))
    for bad in (lambda: ptc.dropout(x, 0.1, 1), lambda: ptc.dropout(y, 0.1, 1, residual=x),
                lambda: ptc.dropout(y, 0.1, 1, out=x), lambda: ptc.quantize_fp4(x),
                lambda: ptc.quantize_fp4(x, transposed="both"), lambda: ptc.matmul_a16_fp4(x, w),
                lambda: ptc.matmul_fp4(w, w, out=torch.zeros(32, 32, device=DEV, requires_grad=True)),
                lambda: ptc.dequantize_fp4(w, out=torch.zeros(32, 64, device=DEV, requires_grad=True))):
        with pytest.raises(RuntimeError, match="requires grad"):
            bad()
    with torch.no_grad():
        want = ptc.dropout(x.detach(), 0.1, 1)
        assert torch.equal(ptc.dropout(x, 0.1, 1), want) and not want.requires_grad
        ptc.quantize_fp4(x)
        ptc.matmul_a16_fp4(x, w)
    assert torch.equal(ptc.dropout(x.detach(), 0.1, 1), want)


def test_results_written_in_place_advance_their_version():
    x = torch.randn(4, 64, device=DEV).bfloat16()
    w = ptc.quantize_fp4(torch.randn(32, 64, device=DEV))
    outs = [x.clone(), torch.empty(4, 32, dtype=torch.bfloat16, device=DEV), torch.empty(32, 32, device=DEV),
            torch.empty(32, 64, device=DEV)]
    before = [t._version for t in outs]
    ptc.dropout(x, 0.5, 1, out=outs[0])
    ptc.matmul_a16_fp4(x, w, out=outs[1])
    ptc.matmul_fp4(w, w, out=outs[2])
    ptc.dequantize_fp4(w, out=outs[3])
    assert all(t._version > b for t, b in zip(outs, before))
    a = torch.ones(4, 64, device=DEV, requires_grad=True)
    saved = a.detach().clone()
    loss = (a * saved).sum()  # autograd keeps `saved` for a's gradient
    ptc.dropout(saved, 0.5, 1, out=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        x = torch.ones(4, 64, device=DEV)
        assert ptc.dropout(x, 0.0, 1, out=x) is x
    out = ptc.dropout(x, 0.0, 1, out=x)
    assert out is x and torch.equal(ptc.dropout(torch.ones(4, 64, device=DEV), 0.0, 1), torch.ones(4, 64, device=DEV))


def test_the_linear_layer_takes_parameters():
    """Its backward pass is explicit, so parameters and activations of a graph may come as they are."""
    x = torch.randn(64, 96, device=DEV).bfloat16()
    w = torch.randn(32, 96, device=DEV).bfloat16()
    dy = torch.randn(64, 32, device=DEV).bfloat16()
    y, saved = fp4_linear.forward(x, w, 0.1, 2, 3)
    want = (y, *fp4_linear.backward(dy, saved))
    y, saved = fp4_linear.forward(x.clone().requires_grad_(), torch.nn.Parameter(w.clone()), 0.1, 2, 3)
    got = (y, *fp4_linear.backward(dy.clone().requires_grad_(), saved))
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not a.requires_grad


def test_a_matrix_of_more_values_than_any_call_takes_is_refused():
    q = ptc.quantize_fp4(torch.ones(4, 64, device=DEV))
    for K in (2 ** 30 + 1, 2 ** 62, 2 ** 63 - 1):
        with pytest.raises(ValueError):
            ptc.Fp4Matrix(q.codes, q.scales, K)
