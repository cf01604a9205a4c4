"""Every launch shape of the 4-bit products, each forced by its key and asserted to be the one that ran.

The reference is a float64 product on the device of the operands' values
(ptc.dequantize_fp4, compared elsewhere for every code and scale).  Bound: the
FP32 sum of K exact products is off by at most (ceil(K / 16) + 4) times 2^-22 of
the sum of magnitudes (twice FP32's truncation of a running sum), and the output
rounding adds one unit roundoff: 2^-24 float32, 2^-8 bfloat16, 2^-11 binary16
(2^-25 absolute for its subnormals)."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
ROUNDOFF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
KEYS = ("fp4_tile", "fp4_ksplit", "fp4_tokens_rows", "fp4_tokens_split")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.fixture(autouse=True)
def keys():
    yield
    for k in KEYS:
        ptc.ptc_set_tuning(k, 0)


def operand(rows, K, fmt, seed, g=None):
    """(Fp4Matrix, float64 values): random codes, block scales within a factor of four (nvfp4: sixteen steps)."""
    gen = torch.Generator(DEV).manual_seed(seed)
    width, block = 16 * -(-K // 32), 16 if fmt == "nvfp4" else 32
    codes = torch.randint(0, 256, (rows, width), generator=gen, device=DEV, dtype=torch.uint8)
    codes[:, (K + 1) // 2:] = 0
    if K % 2:
        codes[:, K // 2] &= 15
    lo, hi = (48, 65) if fmt == "nvfp4" else (126, 129)
    scales = torch.randint(lo, hi, (rows, -(-K // block)), generator=gen, device=DEV, dtype=torch.uint8)
    gt = None if g is None else torch.tensor([g], device=DEV)
    q = ptc.Fp4Matrix(codes, ptc.Fp4Matrix.tile_scales(scales), K, fmt, gt)
    return q, ptc.dequantize_fp4(q, torch.float32).double()


def check(C, a, b, K):
    want, size = a @ b.T, a.abs() @ b.abs().T
    tol = (-(-K // 16) + 4) * 2.0 ** -22 * size
    tol = tol + (want.abs() + tol) * ROUNDOFF[C.dtype] + (2.0 ** -25 if C.dtype == torch.float16 else 0.0)
    off = (C.double() - want).abs()
    assert bool((off <= tol).all()), f"largest error / bound {(off / tol.clamp(min=1e-300)).max().item():.3g}"


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ two 4-bit matrices
# Output tiles beyond two per CTA (pair): each accumulator is used again; K spans more stages than the ring.
MANY = {256: (2600, 3725), 128: (2700, 2100), 64: (2700, 1050)}


@pytest.mark.parametrize("off,ld", [(0, 32), (8, 8), (4, 4), (1, 1)], ids=["wide", "8", "4", "unaligned"])
@pytest.mark.parametrize("dtype", list(ROUNDOFF), ids=str)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("tile", [64, 128, 256])
def test_tiles_that_reuse_both_accumulators(tile, fmt, dtype, off, ld):
    M, N = MANY[tile]
    K = 2400
    ptc.ptc_set_tuning("fp4_tile", tile)
    ptc.ptc_set_tuning("fp4_ksplit", 1)
    A, a = operand(M, K, fmt, 1, 0.7 if fmt == "nvfp4" else None)
    B, b = operand(N, K, fmt, 2)
    pitch = -(-(N + 1) // ld) * ld + (2 if ld == 1 else 0)
    pitch += 1 if ld == 1 and pitch % 2 == 0 else 0
    buf = torch.full((M * pitch + 64,), 7.0, dtype=dtype, device=DEV)
    C = buf[off:off + M * pitch].view(M, pitch)[:, :N]
    ptc.matmul_fp4(A, B, out=C)
    grid, cluster, split, cols = ptc.ptc_last_fp4_launch()
    ctas = 2 if tile == 256 else 1
    tiles = -(-M // (128 * ctas)) * -(-N // tile)
    assert (cluster, split, cols) == (ctas, 1, tile) and tiles > 2 * (grid // ctas) and -(-K // 256) > 8
    check(C, a, b, K)
    buf[off:off + M * pitch].view(M, pitch)[:, :N] = 7.0
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("tile,split", [(t, k) for t in (64, 128) for k in (1, 2, 4, 8)])
@pytest.mark.parametrize("M,N,K", [(64, 512, 8192), (130, 200, 2048), (300, 333, 5000), (1, 64, 2049)])
def test_k_shared_in_clusters(M, N, K, tile, split, fmt):
    ptc.ptc_set_tuning("fp4_tile", tile)
    ptc.ptc_set_tuning("fp4_ksplit", split)
    A, a = operand(M, K, fmt, 3)
    B, b = operand(N, K, fmt, 4)
    for dt in ROUNDOFF:
        C = ptc.matmul_fp4(A, B, out_dtype=dt)
        assert ptc.ptc_last_fp4_launch()[1:] == (split, split, tile)
        check(C, a, b, K)


@pytest.mark.parametrize("M,N,K,want", [(512, 512, 512, (1, 64)), (64, 512, 8192, (8, 64)), (2048, 2048, 2048, (1, 256)),
                                        (1024, 1344, 2090, (1, 128)), (4096, 8192, 2048, (1, 256))])
def test_shapes_taken_by_size(M, N, K, want):
    """The shapes that the measured figures are quoted for, and their results."""
    if sms() != 152:
        pytest.skip("the estimate is made for 152 SMs")
    A, a = operand(M, K, "mxfp4", 5)
    B, b = operand(N, K, "mxfp4", 6)
    C = ptc.matmul_fp4(A, B)
    assert ptc.ptc_last_fp4_launch()[2:] == want
    check(C, a, b, K)


# ------------------------------------------------------------------ few tokens
SHAPES = [(R, M) for R, Ms in ((1, (1, 6)), (2, (1, 8, 12)), (4, (1, 8, 16)), (8, (1, 7, 16, 21))) for M in Ms]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("long", [False, True], ids=["short", "long"])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("R,M", SHAPES)
def test_few_tokens(R, M, split, long, dtype, fmt):
    """All row groups and clusters; K of about one stage per share, and (long) more than its buffer holds, so that two
    buffers of activations take turns; rows of the weights that end inside a tile, activations aligned and not."""
    shares = 8 // R * split
    toks = min(M, 8 if M <= 8 else 16)
    held = 28 * 1024 // (8 // R * (toks * 512 + (256 if M <= 8 else 512)))  # stages of a buffer, at least
    K = 256 * shares * ((held + 4) if long else 1) + 77
    N = 200
    ptc.ptc_set_tuning("fp4_tokens_rows", R)
    ptc.ptc_set_tuning("fp4_tokens_split", split)
    W, w = operand(N, K, fmt, 7, 0.3 if fmt == "nvfp4" else None)
    gen = torch.Generator(DEV).manual_seed(8)
    big = (torch.randn(M, K + 11, generator=gen, device=DEV) * 0.05).to(dtype)
    for x in (big[:, 3:3 + K], torch.nn.functional.pad(big, (0, -(K + 11) % 8))[:, :K]):
        C = ptc.matmul_a16_fp4(x, W)
        grid, cluster, ks, rows = ptc.ptc_last_fp4_launch()
        assert (cluster, ks, rows) == (split, split, 16 * R) and grid == 2 * (8 // R) * split * (2 if M > 16 else 1)
        check(C, x.double(), w, K)


@pytest.mark.parametrize("M,N,K,fmt,dtype", [(1, 4096, 4096, "mxfp4", torch.bfloat16),
                                                  (8, 4096, 4096, "mxfp4", torch.float16),
                                                  (16, 8192, 8192, "mxfp4", torch.bfloat16),
                                                  (16, 16384, 8192, "nvfp4", torch.float16),
                                                  (1, 16384, 8192, "mxfp4", torch.bfloat16)])
def test_few_tokens_at_the_sizes_of_the_measured_figures(M, N, K, fmt, dtype):
    W, w = operand(N, K, fmt, 9)
    x = (torch.randn(M, K, generator=torch.Generator(DEV).manual_seed(10), device=DEV) * 0.05).to(dtype)
    C = ptc.matmul_a16_fp4(x, W)
    check(C, x.double(), w, K)


def test_a_shape_that_does_not_fit_is_not_taken():
    W, w = operand(200, 300, "mxfp4", 11)
    x = torch.randn(3, 300, generator=torch.Generator(DEV).manual_seed(12), device=DEV).half()
    ptc.matmul_a16_fp4(x, W)
    by_size = ptc.ptc_last_fp4_launch()
    ptc.ptc_set_tuning("fp4_tokens_rows", 1)
    ptc.ptc_set_tuning("fp4_tokens_split", 8)
    C = ptc.matmul_a16_fp4(x, W)
    assert ptc.ptc_last_fp4_launch() == by_size  # 300 of K are two stages, no 64 shares
    check(C, x.double(), w, 300)
