"""Calls of the 4-bit products that give up: the status is reported, the call ends
within a few wait limits, and the calls after it are right.

The first operands of a tile are withheld (a test hook of the library); later
stages of the ring are loaded and are waited for before the CTA exits."""
import time

import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
LIMIT_NS = 3_000_000


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def held(rows, K, fmt, seed):
    x = torch.randn(rows, K, generator=torch.Generator(DEV).manual_seed(seed), device=DEV)
    return ptc.quantize_fp4(x, fmt)


def gives_up_and_recovers(call):
    want = call()
    torch.cuda.synchronize()
    try:
        for tile in (0, 1):
            ptc.ptc_debug_set_wait_limit(LIMIT_NS, tile)
            t = time.monotonic()
            call()
            torch.cuda.synchronize()
            assert time.monotonic() - t < 0.5
            assert ptc.gemm_poll_device_error() == ptc.PTC_ERR_TIMEOUT
            ptc.ptc_debug_set_wait_limit(0, -1)
            for _ in range(3):
                assert torch.equal(call(), want)
            assert ptc.gemm_poll_device_error() == ptc.PTC_OK
    finally:
        ptc.ptc_debug_set_wait_limit(0, -1)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("tile,split", [(64, 1), (64, 4), (64, 8), (128, 1), (128, 2), (256, 1)])
def test_product(tile, split, fmt):
    A, B = held(600, 6000, fmt, 1), held(520, 6000, fmt, 2)  # 24 stages, three times the ring
    ptc.ptc_set_tuning("fp4_tile", tile)
    ptc.ptc_set_tuning("fp4_ksplit", split)
    try:
        gives_up_and_recovers(lambda: ptc.matmul_fp4(A, B))
    finally:
        ptc.ptc_set_tuning("fp4_tile", 0)
        ptc.ptc_set_tuning("fp4_ksplit", 0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 300, 9000), (5, 1000, 600)])
def test_few_tokens(M, N, K, fmt):
    W = held(N, K, fmt, 3)
    x = torch.randn(M, K, generator=torch.Generator(DEV).manual_seed(4), device=DEV).bfloat16()
    gives_up_and_recovers(lambda: ptc.matmul_a16_fp4(x, W))
