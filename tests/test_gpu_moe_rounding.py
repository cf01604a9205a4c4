"""What the rounding of h, the experts' intermediate activations, costs: codes are held as n = c + 8, and
what (8 + z) takes off again has to be the sum of the numbers that n multiplied."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.s4_ref import gen, matrix, rand, weights

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("inner, at", [(32, 0), (32, 31), (200, 130), (200, 135), (256, 77)])
def test_weights_of_zero_give_zero(inner, at, group, dtype):
    """One h that is not zero and has more bits than are kept, weights of code 0: n is 8 for all of them, one
    product stands against one sum, and both are exact in FP32."""
    D = 48
    groups = -(-D // group)
    up = torch.zeros(1, 2 * inner, 32, device=DEV, dtype=torch.uint8)
    up[0, at, 0] = 7          # gate 7 x
    up[0, inner + at, 0] = 3  # up 3 x
    one = torch.ones(1, 2 * inner, groups, device=DEV, dtype=dtype)
    down = torch.zeros(1, D, -(-inner // 32) * 16, device=DEV, dtype=torch.uint8)
    two = torch.ones(1, D, -(-inner // group), device=DEV, dtype=dtype)
    S = ptc.S4Matrix.tile_scales
    x = torch.zeros(3, D, device=DEV, dtype=dtype)
    x[:, 0] = torch.tensor([0.71, 1.0, 1.37], device=DEV)
    y = ptc.moe_a16_s4(x, torch.zeros(1, D, device=DEV, dtype=dtype), ptc.S4Matrix(up, S(one), D, group),
                       ptc.S4Matrix(down, S(two), inner, group), 1)
    assert not y.any(), y.abs().max()


@pytest.mark.parametrize("T, D, I, E, k", [(16, 1024, 512, 8, 4), (8, 512, 1024, 4, 2)])
@pytest.mark.parametrize("group", [32, 128])
def test_error_beside_that_of_y(T, D, I, E, k, group):
    """bfloat16: y's own rounding is off by 2^-9 of an element at most, h's (11 bits) by 2^-12 of an element:
    an eighth.  Errors of h reach y weighted as h itself does, and independent of it, so that the norm of y's error is
    sqrt(1 + 1 / 64) = 1.008 times that of rounding y alone; the FP32 sums add less than 2^-13 of y, 0.001 times
    that.  With codes of -3 .. 3 (n = c + 8 is four times c in the mean square) a sum of other numbers than those
    multiplied gives sqrt(1 + (4.1 / 8)^2) = 1.12.  T D errors: the norms' quotient varies by 0.005."""
    gu, dn = weights(1, (E,), 2 * I, D, group), weights(2, (E,), D, I, group)
    for w, seed, n in ((gu, 3, D), (dn, 4, I)):
        c = torch.randint(-3, 4, (E, w["scales"].shape[1], -(-n // 32) * 32), generator=gen(seed), device=DEV)
        nib = (c & 15).to(torch.uint8)
        w["codes"] = (nib[..., 0::2] | (nib[..., 1::2] << 4)).contiguous()
        w["scales"] = (0.5 * n ** -0.5 * (1 + torch.rand(w["scales"].shape, generator=gen(seed + 9), device=DEV))).to(BF)
        w["values"] = c[..., :n].double() * w["scales"].double()[..., torch.arange(n, device=DEV) // group]
    x, router = rand(5, T, D, dtype=BF), rand(6, E, D, dtype=BF, size=D ** -0.5)
    y, ids, p = ptc.moe_a16_s4(x, router, matrix(gu), matrix(dn), k, return_routing=True)
    want = torch.zeros(T, D, device=DEV, dtype=torch.float64)
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        g, u = (x[tok].double() @ gu["values"][e].t()).split(I, 1)
        want.index_add_(0, tok, p[tok, slot].double().unsqueeze(1) * ((g * torch.sigmoid(g) * u) @ dn["values"][e].t()))
    rounding = (want.to(BF).double() - want).norm()
    assert (y.double() - want).norm() <= 1.03 * rounding, ((y.double() - want).norm() / rounding)
