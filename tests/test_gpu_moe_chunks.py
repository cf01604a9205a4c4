"""The experts' sums of chunks: more chunks than one per stage of codes would give, more tiles of rows than
places, and each of them against the formula, twice the same."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.test_gpu_moe import compare, layer, run

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("T, D, I, E, k, group, dtype", [
    (1, 64, 70000, 2, 1, 128, BF),    # 274 stages in 137 chunks of two
    (3, 96, 30000, 3, 2, 32, HF),     # 118 stages in 40 chunks of three, the last of one
    (1, 17000, 40, 3, 2, 64, BF),     # 532 tiles of rows, 512 places
    (9, 20011, 300, 4, 2, 128, HF),   # the same with several items per CTA and ragged ends
    (64, 16417, 64, 16, 8, 32, BF),   # 514 tiles, 512 pairs
    (64, 300, 2000, 16, 8, 256, HF),  # 512 pairs, one chunk of eight stages each
])
def test_chunks_and_places(T, D, I, E, k, group, dtype):
    L = layer(500 + T, T, D, I, E, k, group, group == 32, dtype)
    got = run(L)
    compare(L, got)
    for a, b in zip(run(L), got):
        assert torch.equal(a, b)
