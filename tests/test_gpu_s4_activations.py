"""The activations as the grouped 4-bit product holds them, one by one."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.s4_ref import gen

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("dtype, exact", [(BF, -27), (HF, -24)])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("largest", [2.0 ** 15, 1.9375 * 2.0 ** 15])
def test_one_by_one(largest, group, dtype, exact):
    """With codes of -8 and zeros of -8 every weight is 0, its n and its (8 + z) too; one code of -7 per row gives that
    row's element as it is held, through exact products and sums of one number.  Elements of every mantissa bit, at
    every place of a block, from the largest down to 2^-34 of it: exact down to 2^exact of it, off by at most 2^-35
    of it below (and half a step of the result's type)."""
    K, M = 256, 16
    c = torch.full((K, K), 8, device=DEV, dtype=torch.uint8)  # -8
    c.fill_diagonal_(9)                                       # -7
    codes = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
    one = torch.ones(K, -(-K // group), device=DEV, dtype=dtype)
    S = ptc.S4Matrix.tile_scales
    m = ptc.S4Matrix(codes, S(one), K, group, S(-8 * one))
    block = min(group, 128)
    for seed in range(6):
        g = gen(seed)
        mantissa = 1 + torch.rand(M, K, generator=g, device=DEV)
        e = -torch.rand(M, K, generator=g, device=DEV) * 34
        x = (largest * torch.exp2(e.floor()) * mantissa.clamp(max=1.99) / 2).to(dtype)
        x = torch.where(torch.rand(M, K, generator=g, device=DEV) < 0.5, -x, x)
        x[:, seed::block] = largest
        y = ptc.matmul_a16_s4(x, m)
        v, off = x.double(), (y.double() - x.double()).abs()
        kept = v.abs() >= 2.0 ** exact * largest
        assert not off[kept].any()
        t = torch.finfo(dtype)
        assert bool((off <= 2.0 ** -35 * largest + t.eps / 2 * v.abs() + t.smallest_normal * t.eps).all())
        assert int((~kept).sum()) > 100  # (both are seen)
