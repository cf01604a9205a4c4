"""The experts' choice at its edges: logits that are zeros of both signs, and sizes that are refused."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.s4_ref import matrix, rand, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def experts(E, D=64, I=32):
    return matrix(weights(1, (E,), 2 * I, D, 32)), matrix(weights(2, (E,), D, I, 32))


@pytest.mark.parametrize("E", [5, 70, 130])
def test_zeros_of_both_signs_are_equal(E):
    """A logit of products that are all negative and too small for FP32 is -0, which is as large as +0: the lowest
    index first.  (2048 columns: a thread without columns would add its +0.)"""
    D = 2048
    gu, dn = experts(E, D)
    x = torch.full((2, D), -2.0 ** -100, device=DEV, dtype=torch.bfloat16)
    router = torch.zeros(E, D, device=DEV)
    router[0] = router[3] = 2.0 ** -100
    logits = x.float() @ router.t()
    assert not logits.any()
    _, ids, p = ptc.moe_a16_s4(x, router, gu, dn, 4, return_routing=True)
    assert ids.tolist() == [[0, 1, 2, 3]] * 2 and bool((p == 0.25).all())


def test_a_top_k_beyond_all_experts_is_refused():
    """Before anything of its size is allocated."""
    gu, dn = experts(6)
    x, router = rand(3, 4, 64, dtype=torch.bfloat16), rand(4, 6, 64, dtype=torch.bfloat16)
    for top_k in (7, 10 ** 12, 2 ** 62):
        for tokens in (x, x[:0]):
            with pytest.raises(ptc.PtcError):
                ptc.moe_a16_s4(tokens, router, gu, dn, top_k, return_routing=True)
