"""The few-token product over the whole exponent range of its activations and scales.

Bound: the FP32 sum of K exact products is off by at most (ceil(K / 16) + 4) times
2^-22 of the sum of magnitudes, and the output rounding adds one unit roundoff
(2^-8 bfloat16, 2^-11 binary16)."""
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


def weights(codes, byte, K, fmt="mxfp4"):
    q = ptc.Fp4Matrix(torch.from_numpy(ref.pack(codes, 16 * -(-K // 32))).to(DEV), torch.from_numpy(ref.tile(byte)).to(DEV),
                      K, fmt)
    return q, ref.values(codes, byte, K, fmt)


def check(C, x, w, K):
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = (-(-K // 16) + 4) * 2.0 ** -22 * size
    tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    off = np.abs(C.cpu().double().numpy() - want)
    assert np.isfinite(want).all() and np.all(off <= tol), f"{np.sum(~(off <= tol))} of {off.size}"


@pytest.mark.parametrize("value,code,byte", [(1e37, 7, 107), (6e37, 7, 107), (3.3e38, 7, 0), (3.3e38, 1, 110), (-3e38, 7, 90)])
@pytest.mark.parametrize("M,N,K", [(1, 128, 32), (3, 40, 96), (16, 257, 2048)])
def test_largest_bfloat16_with_small_scales(M, N, K, value, code, byte):
    """Activations near the type's largest value times weights far below one: each block's sum without its scale is beyond FP32."""
    x = torch.full((M, K), value, dtype=torch.bfloat16, device=DEV)
    W, w = weights(np.full((N, K), code), np.full((N, K // 32), byte), K)
    check(ptc.matmul_a16_fp4(x, W), x.cpu().double().numpy(), w, K)


@pytest.mark.parametrize("M,N,K", [(1, 130, 640), (5, 64, 1024), (8, 300, 4096), (16, 200, 3000)])
def test_blocks_whose_exponents_cancel(M, N, K):
    """Token blocks over bfloat16's whole range against block scales that bring every product back to ordinary size."""
    rng = np.random.default_rng(K)
    blocks = -(-K // 32)
    e = rng.integers(-110, 125, blocks)  # of each block, both in x and (negated) in the scales
    x = rng.standard_normal((M, 32 * blocks)) * np.repeat(np.exp2(e.astype(np.float64)), 32)
    x = torch.from_numpy(x[:, :K].astype(np.float32)).to(torch.bfloat16).to(DEV)
    byte = np.clip(127 - e + rng.integers(-2, 3, (N, blocks)), 0, 254)
    codes = np.zeros((N, 32 * blocks), dtype=np.int64)
    codes[:, :K] = rng.integers(0, 16, (N, K))
    W, w = weights(codes, byte, K)
    check(ptc.matmul_a16_fp4(x, W), x.cpu().double().numpy(), w, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("top", [1.0, 1.5, 255 / 128])
def test_small_activations_beside_a_large_one(fmt, top):
    """Elements down to 2^-32 of the largest of their 32 are exact (eight significant bits each)."""
    K, n = 256, ref.BLOCK[fmt]
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (64, K))
    codes[:, ::32] = 0  # the large element's weight
    W, w = weights(codes, np.full((64, K // n), 127 if fmt == "mxfp4" else 56), K, fmt)
    x = np.zeros((4, K))
    x[:, ::32] = top
    x[np.arange(4)[:, None], np.arange(8) * 32 + 1 + rng.integers(0, 31, (4, 8))] = rng.integers(129, 256, (4, 8)) * 2.0 ** -39
    x = x * np.array([1.0, 2.0 ** 60, 2.0 ** -60, -8.0])[:, None]
    C = ptc.matmul_a16_fp4(torch.from_numpy(x.astype(np.float32)).bfloat16().to(DEV), W)
    want = torch.from_numpy((x @ w.T).astype(np.float32)).bfloat16()  # few terms of 12 bits: exact in FP32
    assert torch.equal(C.cpu(), want)
