"""The norms at their edges."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("rows", [1, 4, 1000])
def test_s8_rows_of_no_values_have_scale_zero(rows):
    """As rows of zeros have: the INT8 product that takes the scales is then 0, not what memory held."""
    scale = torch.full((rows,), float("nan"), device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    ptc.ptc_rms_norm_s8(rows, 0, None, 0, ptc.PTC_OUT_BF16, None, 0, None, 0, None, ptc.PTC_OUT_BF16, 1e-6, None, 0,
                        scale.data_ptr(), stream)
    assert not scale.any()
    for residual in (False, True):
        x = torch.empty(rows, 0, device=DEV, dtype=torch.bfloat16)
        torch.cuda.synchronize()
        dirty = [torch.full((rows,), float("nan"), device=DEV) for _ in range(8)]
        del dirty
        got = ptc.rms_norm_s8(x, residual=x.clone() if residual else None)
        assert got[0].shape == (rows, 0) and got[1].shape == (rows,) and not got[1].any()
    with pytest.raises(ptc.PtcError):
        ptc.ptc_rms_norm_s8(rows, 0, None, 0, ptc.PTC_OUT_BF16, None, 0, None, 0, None, ptc.PTC_OUT_BF16, 1e-6, None, 0, None, stream)


def test_dweight_of_many_small_rows_beside_a_large_one():
    """One row of 1 and 37 of 2^-24, among 300 that are all partial sums of their own: every sum of theirs passes
    through at most 9 + 2 + 3 additions, each off by half an ulp.  (Added one after the other, all 37 are lost.)"""
    rows, cols = 300, 64
    dy = torch.zeros(rows, cols, device=DEV)
    dy[::8] = 2.0 ** -24
    dy[0] = 1.0
    _, dw = ptc.rms_norm_backward(dy, torch.ones(rows, cols, device=DEV), eps=0.0)
    want = dy.double().sum(0)
    assert bool(((dw.double() - want).abs() <= 15 * 2.0 ** -24 * want).all()), ((dw.double() - want) * 2.0 ** 24)[0]
