"""The grouped 4-bit product after a wait that runs out, with operands made beforehand that come in several chunks:
nothing more is brought, what is on its way lands, the status says so, and the next call is whole."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.s4_ref import check, matrix, rand, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    for k in ("s4_tokens_rows", "s4_tokens_split"):
        ptc.ptc_set_tuning(k, 0)
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("rows, split", [(1, 1), (16, 1), (4, 2), (1, 8)])
@pytest.mark.parametrize("M, N, K", [(16, 3000, 70000), (16, 6000, 4096), (3, 400, 40000)])
def test_with_operands_in_chunks(M, N, K, rows, split):
    w = weights(1, (), N, K, 128, False, torch.bfloat16)
    m, x = matrix(w), rand(2, M, K, dtype=torch.bfloat16)
    assert ptc.gemm_a16_s4_workspace(M, K) > 0 and M * -(-K // 256) > 64
    ptc.ptc_set_tuning("s4_tokens_rows", rows)
    ptc.ptc_set_tuning("s4_tokens_split", split)
    want = ptc.matmul_a16_s4(x, m)
    check(want, x, w, torch.bfloat16)
    torch.cuda.synchronize()
    ptc.ptc_debug_set_wait_limit(20_000_000, 1)
    try:
        ptc.matmul_a16_s4(x, m)
        torch.cuda.synchronize()
        assert ptc.lib().gemm_poll_device_error() == ptc.PTC_ERR_TIMEOUT
    finally:
        ptc.ptc_debug_set_wait_limit(0, -1)
    for _ in range(3):
        assert torch.equal(ptc.matmul_a16_s4(x, m), want)
