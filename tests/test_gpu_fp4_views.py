"""Results beside their inputs in one buffer: column slices that share rows of memory but no byte."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,at", [(64, 64), (63, 63), (40, 104), (1, 1)])
def test_dropout_between_columns_of_one_buffer(cols, at, dtype):
    buf = torch.randn(50, 168, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    first = buf.clone()
    want = torch.from_numpy(ref.dropout(first[:, :cols].cpu().float().numpy(), 0.3, 5, 6)).to(dtype)
    ptc.dropout(buf[:, :cols], 0.3, 5, 6, out=buf[:, at:at + cols])
    assert torch.equal(buf[:, at:at + cols].cpu(), want)
    buf[:, at:at + cols] = first[:, at:at + cols]
    assert torch.equal(buf, first)
    # the other way round, with what lies there as the residual
    want = torch.from_numpy(ref.dropout(first[:, at:at + cols].cpu().float().numpy(), 0.3, 5, 6,
                                        first[:, :cols].cpu().float().numpy())).to(dtype)
    ptc.dropout(buf[:, at:at + cols], 0.3, 5, 6, residual=buf[:, :cols], out=buf[:, :cols])
    assert torch.equal(buf[:, :cols].cpu(), want) and torch.equal(buf[:, cols:], first[:, cols:])


def test_few_tokens_between_columns_of_one_buffer():
    W = ptc.quantize_fp4(torch.randn(96, 160, generator=torch.Generator().manual_seed(3)).to(DEV))
    buf = torch.randn(7, 264, generator=torch.Generator().manual_seed(4)).bfloat16().to(DEV)
    first = buf.clone()
    want = ptc.matmul_a16_fp4(first[:, :160], W)
    ptc.matmul_a16_fp4(buf[:, :160], W, out=buf[:, 160:256])
    assert torch.equal(buf[:, 160:256], want) and torch.equal(buf[:, :160], first[:, :160])
    assert torch.equal(buf[:, 256:], first[:, 256:])


def test_overlapping_columns_are_still_refused():
    buf = torch.zeros(20, 100, dtype=torch.bfloat16, device=DEV)
    for a, b in (((0, 40), (39, 79)), ((40, 100), (0, 60)), ((0, 50), (49, 99))):
        with pytest.raises(ptc.PtcError):
            ptc.dropout(buf[:, slice(*a)], 0.1, 1, out=buf[:, slice(*b)])
    wrap = buf.view(-1)[50:1950].view(19, 100)  # its rows are the second halves of buf's rows and the first halves of the next ones
    with pytest.raises(ptc.PtcError):
        ptc.dropout(buf[:19, :60], 0.1, 1, out=wrap[:, :60])
    with pytest.raises(ptc.PtcError):  # other pitches: whole spans are compared
        ptc.dropout(buf[:10, :40], 0.1, 1, out=buf[::2, 40:80])
