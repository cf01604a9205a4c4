"""A token's result through the experts, whatever the other tokens of the call are."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.test_gpu_moe import layer, run

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("T, D, I, E, k, group, dtype", [(16, 1024, 512, 32, 4, 128, HF), (9, 256, 64, 20, 3, 64, BF), (33, 500, 1300, 10, 5, 32, HF),
                                                         (64, 512, 256, 128, 8, 128, HF), (4, 2048, 768, 40, 8, 256, BF)])
def test_other_tokens_do_not_matter(T, D, I, E, k, group, dtype):
    """Other tokens choose other experts, which moves the work between warps and CTAs: every sum's order stays."""
    for seed in range(4):
        L = layer(400 + seed, T, D, I, E, k, group, False, dtype)
        want = run(L)
        keep = torch.arange(T, device=DEV) % 4 == seed
        L["x"] = torch.where(keep.unsqueeze(1), L["x"], L["x"].flip(1))
        L["x"][~keep, 3] = float("nan") if seed == 3 else 1.0
        got = run(L)
        assert not torch.equal(got[1], want[1])
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep]), seed
