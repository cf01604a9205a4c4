"""GPU parity of counter-based dropout, microscaled 4-bit quantisation and the
4-bit products with the plain 64-bit reference in tests/fp4_ref.py.

Bounds.  Dropout and quantisation are functions of their inputs to the last
bit, so codes, scale bytes and values are compared for equality (a zero's sign
aside).  A product's FP32 sum of K exact terms is off its exact value by at most
(ceil(K / 16) + 4) additions' errors of 2^-22 of the sum of magnitudes each
(twice FP32's 2^-23 relative truncation of a running sum), and the output
rounding adds half a unit in the last place (2^-9, 2^-12 or 2^-24 relative,
2^-25 absolute for binary16 subnormals)."""
import numpy as np
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from precision_tensor_core_gb300 import fp4_linear
from tests import fp4_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12}
SEED, OFFSET = 0x9E3779B97F4A7C15, (5 << 32) + 77


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.fixture(params=[(64, 1), (64, 4), (128, 1), (128, 2), (256, 1), (0, 0)], ids=lambda p: f"tile{p[0]}ks{p[1]}")
def shape(request):
    ptc.ptc_set_tuning("fp4_tile", request.param[0])
    ptc.ptc_set_tuning("fp4_ksplit", request.param[1])
    yield request.param
    ptc.ptc_set_tuning("fp4_tile", 0)
    ptc.ptc_set_tuning("fp4_ksplit", 0)


def host(t):
    return t.detach().cpu().double().numpy()


def f32(t):
    return t.detach().cpu().float().numpy()


def normal(rows, cols, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(1, cols, generator=g))
    return x.to(dtype).to(DEV)


def rounded(y, dtype):
    """An FP32 numpy result rounded to a torch dtype, as float64."""
    return host(torch.from_numpy(np.ascontiguousarray(y, dtype=np.float32)).to(dtype))


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


# ------------------------------------------------------------------ dropout
SHAPES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 64), (33, 1000), (130, 257), (1, 4096)]


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout(rows, cols, dtype, residual):
    x = normal(rows, cols, 1, DT[dtype], 0.5)
    r = normal(rows, cols, 2, DT[dtype], 0.5) if residual else None
    y = ptc.dropout(x, 0.3, SEED, OFFSET, residual=r)
    want = ref.dropout(f32(x), 0.3, SEED, OFFSET, None if r is None else f32(r))
    assert y.dtype == x.dtype and same(host(y), rounded(want, x.dtype))


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.5, 0.9999, 1.0])
def test_dropout_probabilities(p):
    x = normal(64, 1024, 3, torch.float32, 0.1)
    y = ptc.dropout(x, p, 12345, 0)
    assert same(host(y), rounded(ref.dropout(f32(x), p, 12345, 0), torch.float32))
    if p == 0.0:
        assert torch.equal(y, x)
    if p == 1.0:
        assert not y.any()


def test_dropout_strides_in_place_and_other_streams():
    big = normal(50, 300, 4, torch.bfloat16, 0.5)
    for x in (big[:, 3:200], big[::2, :120], big[5:6, 1:], big[:, 8:136]):
        want = rounded(ref.dropout(f32(x), 0.2, 7, 9), x.dtype)
        assert same(host(ptc.dropout(x, 0.2, 7, 9)), want)
    x = big.clone()
    want = rounded(ref.dropout(f32(x), 0.2, 7, 9, f32(big)), x.dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ptc.dropout(x, 0.2, 7, 9, residual=big, out=x, stream=side)
    side.synchronize()
    assert y is x and same(host(x), want)


def test_dropout_drops_infinities_and_keeps_them():
    x = torch.full((16, 64), float("inf"), device=DEV)
    x[::2] = float("nan")
    y = host(ptc.dropout(x, 0.5, 1, 2))
    keep = ref.bits16(16, 64, 1, 2, 0) < 32768
    assert np.all(y[~keep] == 0) and np.all(np.isinf(y[1::2][keep[1::2]])) and np.all(np.isnan(y[::2][keep[::2]]))


def test_dropout_gradient_is_the_same_call():
    """d(dropout(x).g)/dx by differences (the map is linear: steps of a power of two are exact) and by the formula."""
    x = torch.round(normal(6, 40, 5, torch.float32, 0.0) * 8)
    g = torch.round(normal(6, 40, 6, torch.float32, 0.0) * 8)
    dx = host(ptc.dropout(g, 0.5, SEED, 3))
    keep = ref.bits16(6, 40, SEED, 3, 0) < 32768
    assert same(dx, np.where(keep, 2 * host(g), 0.0))
    base = host(ptc.dropout(x, 0.5, SEED, 3))
    for i, j in [(0, 0), (0, 39), (5, 17), (3, 8), (2, 31)]:
        xp = x.clone()
        xp[i, j] += 0.5
        diff = ((host(ptc.dropout(xp, 0.5, SEED, 3)) - base) * host(g)).sum() / 0.5
        assert diff == dx[i, j]


# ------------------------------------------------------------------ quantisation
def check_quantised(q, x, fmt, rounding, bits, g):
    """Codes and scale bytes of q against the reference of x (FP32 numpy)."""
    codes, byte = ref.quantize(x, fmt, rounding, bits, g)
    width = 16 * -(-x.shape[1] // 32)
    got = ref.unpack(q.codes.cpu().numpy())
    assert q.codes.shape == (x.shape[0], width)
    want = ref.unpack(ref.pack(codes, width))
    got = np.where(got == 8, 0, got)  # a rounded-away negative keeps its sign
    assert np.array_equal(got, want)
    assert np.array_equal(q.row_scales().cpu().numpy(), byte)
    # whole tiles: rows past the last and blocks past K are zero
    tiles = q.scales.cpu().numpy()
    assert tiles.size == ptc.fp4_scale_bytes(*x.shape, fmt) and np.array_equal(tiles, ref.tile(byte))
    return codes, byte


QSHAPES = [(1, 1), (1, 31), (2, 33), (5, 128), (129, 100), (31, 520), (128, 256), (300, 17), (1, 4096), (257, 129)]


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", QSHAPES)
def test_quantize(rows, cols, dtype, fmt, rounding):
    x = normal(rows, cols, rows + cols, DT[dtype])
    g = (x.float().abs().amax() / 2688).reshape(1) if fmt == "nvfp4" and cols % 2 else None
    gv = None if g is None else np.float32(g.item())
    bits = ref.bits16(rows, cols, SEED, OFFSET, 1) if rounding == "stochastic" else None
    tb = None if bits is None else bits.T
    kw = dict(rounding=rounding, tensor_scale=g, seed=SEED, offset=OFFSET)
    xn = f32(x)
    q = ptc.quantize_fp4(x, fmt, **kw)
    codes, byte = check_quantised(q, xn, fmt, rounding, bits, gv)
    check_quantised(ptc.quantize_fp4(x, fmt, transposed=True, **kw), np.ascontiguousarray(xn.T), fmt, rounding, tb, gv)
    a, b = ptc.quantize_fp4(x, fmt, transposed="both", **kw)
    check_quantised(a, xn, fmt, rounding, bits, gv)
    check_quantised(b, np.ascontiguousarray(xn.T), fmt, rounding, tb, gv)
    # and back: exact products of code and scale, rounded (twice with a matrix scale)
    v = ref.values(codes, byte, cols, fmt).astype(np.float32)
    v = v if gv is None else v * gv
    for dt in DT.values():
        assert same(host(ptc.dequantize_fp4(q, dt)), rounded(v, dt))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_quantize_with_dropout(fmt, rounding):
    x = normal(70, 150, 11, torch.bfloat16)
    g = (x.float().abs().amax() / 2000).reshape(1) if fmt == "nvfp4" else None
    gv = None if g is None else np.float32(g.item())
    xd = ref.dropout(f32(x), 0.25, SEED, 4)
    bits = ref.bits16(70, 150, SEED, 4, 1) if rounding == "stochastic" else None
    tb = None if bits is None else bits.T
    kw = dict(rounding=rounding, tensor_scale=g, p=0.25, seed=SEED, offset=4)
    check_quantised(ptc.quantize_fp4(x, fmt, **kw), xd, fmt, rounding, bits, gv)
    a, b = ptc.quantize_fp4(x, fmt, transposed="both", **kw)
    check_quantised(a, xd, fmt, rounding, bits, gv)
    check_quantised(b, np.ascontiguousarray(xd.T), fmt, rounding, tb, gv)


def test_quantize_ties_limits_and_values_that_are_not_finite():
    row = np.zeros((8, 64), dtype=np.float32)
    row[0, :32] = np.arange(32) * 0.25 - 2  # ties of every gap, scale 1
    row[0, 0] = 6
    row[0, 32:64] = np.array([5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 7.9] * 4)
    row[1, 3] = np.inf
    row[2, 40] = np.nan
    row[3, :] = 1e-45  # the smallest FP32 subnormal
    row[3, 33] = 2.0 ** -126
    row[4, :] = 3.4028235e38
    row[5, ::2] = -0.0
    row[6, 5] = -np.inf
    row[7, :] = 2.0 ** np.linspace(-30, 30, 64)
    x = torch.from_numpy(row).to(DEV)
    for fmt in ("mxfp4", "nvfp4"):
        for rounding in ("nearest", "stochastic"):
            bits = ref.bits16(8, 64, 1, 0, 1) if rounding == "stochastic" else None
            q = ptc.quantize_fp4(x, fmt, rounding=rounding, seed=1)
            check_quantised(q, row, fmt, rounding, bits, None)
            qt = ptc.quantize_fp4(x, fmt, transposed=True, rounding=rounding, seed=1)
            check_quantised(qt, np.ascontiguousarray(row.T), fmt, rounding, None if bits is None else bits.T, None)
        v = host(ptc.dequantize_fp4(ptc.quantize_fp4(x, fmt), torch.float32))
        n = ref.BLOCK[fmt]
        assert np.isnan(v[1, :n]).all() and np.isfinite(v[1, 32:]).all() and np.isnan(v[2, 40 // n * n:][:n]).all()


@pytest.mark.parametrize("g", [2.0 ** -100, 1e-20, 1.0, 3.7, 1e20])
def test_quantize_saturates_where_the_matrix_scale_is_small(g):
    x = normal(20, 80, 13, torch.float32, 6.0)
    x[3, 5], x[4, 70], x[5, 16:32] = 3e38, -3e38, 2.0 ** -126
    t = torch.tensor([g], dtype=torch.float32, device=DEV)
    for rounding in ("nearest", "stochastic"):
        bits = ref.bits16(20, 80, 2, 0, 1) if rounding == "stochastic" else None
        q = ptc.quantize_fp4(x, "nvfp4", rounding=rounding, tensor_scale=t, seed=2)
        check_quantised(q, f32(x), "nvfp4", rounding, bits, np.float32(t.item()))


def test_quantize_ties_of_nvfp4_scales():
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    d = ref.E4M3[8:].astype(np.float32)[:, None]
    x = np.concatenate([6 * d, mid * d, np.zeros((d.shape[0], 8), np.float32)], axis=1)
    check_quantised(ptc.quantize_fp4(torch.from_numpy(x).to(DEV), "nvfp4"), x, "nvfp4", "nearest", None, None)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_stochastic_thresholds(fmt):
    """Values where the code goes up for the element's own random number, and their FP32 neighbours."""
    bits = ref.bits16(128, 96, SEED, 5, 1)
    rng = np.random.default_rng(3)
    low = rng.integers(0, 7, bits.shape)
    x = (ref.GRID[low] + (ref.GRID[low + 1] - ref.GRID[low]) * (65536 - bits) / 65536).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, x.shape).astype(np.int32)).view(np.float32)
    x = np.minimum(x, np.float32(6)) * rng.choice(np.float32([-1, 1]), x.shape)
    x[np.add.outer(np.arange(128), np.arange(96)) % 16 == 0] = 6  # in every block: its scale is 1
    a, b = ptc.quantize_fp4(torch.from_numpy(x).to(DEV), fmt, transposed="both", rounding="stochastic", seed=SEED, offset=5)
    check_quantised(a, x, fmt, "stochastic", bits, None)
    check_quantised(b, np.ascontiguousarray(x.T), fmt, "stochastic", bits.T, None)


def test_quantize_strided_input_and_empty():
    big = normal(40, 400, 12, torch.float16, 0.5)
    for x in (big[:, 5:205], big[::3, :64], big[7:8, 2:], big[:, 16:144]):
        check_quantised(ptc.quantize_fp4(x), f32(x), "mxfp4", "nearest", None, None)
        check_quantised(ptc.quantize_fp4(x, transposed=True), np.ascontiguousarray(f32(x).T), "mxfp4", "nearest", None, None)
    q = ptc.quantize_fp4(big[:0])
    assert q.shape == (0, 400) and ptc.dequantize_fp4(q).shape == (0, 400)


def test_stochastic_rounding_has_no_bias():
    """The mean of many roundings of one value is the value within five standard deviations."""
    x = torch.full((1024, 64), 1.3, device=DEV)
    x[:, 0::32] = 6.0  # scale 1
    v = host(ptc.dequantize_fp4(ptc.quantize_fp4(x, rounding="stochastic", seed=99), torch.float32))
    v = v[:, np.arange(64) % 32 != 0]
    assert set(np.unique(v)) == {1.0, 1.5}
    sigma = 0.5 * np.sqrt(0.6 * 0.4 / v.size)
    assert abs(v.mean() - float(np.float32(1.3))) < 5 * sigma


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_dequantize_every_code_and_scale(fmt):
    """Every code with every scale byte (a row per byte), at an offset pitch."""
    byte = np.repeat((np.arange(256) & (0x7F if fmt == "nvfp4" else 0xFF))[:, None], 32 // ref.BLOCK[fmt], axis=1)
    codes = np.tile(np.arange(32) % 16, (256, 1))
    packed = torch.zeros(256, 48, dtype=torch.uint8)
    packed[:, :16] = torch.from_numpy(ref.pack(codes, 16))
    q = ptc.Fp4Matrix(packed.to(DEV), torch.from_numpy(ref.tile(byte)).to(DEV), 32, fmt)
    v = ref.values(codes, byte, 32, fmt)
    with np.errstate(over="ignore"):
        v = v.astype(np.float32)
    for dt in DT.values():
        assert same(host(ptc.dequantize_fp4(q, dt)), rounded(v, dt))


# ------------------------------------------------------------------ products
def matrix(rows, K, fmt, seed, spread=1.0, g=None):
    """(Fp4Matrix, float64 values) of random codes with a spread of scales."""
    rng = np.random.default_rng(seed)
    n = ref.BLOCK[fmt]
    blocks, width = -(-K // n), 16 * -(-K // 32)
    codes = np.zeros((rows, 2 * width), dtype=np.int64)
    codes[:, :K] = rng.integers(0, 16, size=(rows, K))
    mid = 127 if fmt == "mxfp4" else 56
    byte = np.clip(np.round(mid + spread * rng.standard_normal((rows, blocks)) * (1 if fmt == "mxfp4" else 8)), 0,
                   254 if fmt == "mxfp4" else 126).astype(np.int64)
    gt = None if g is None else torch.tensor([g], dtype=torch.float32, device=DEV)
    q = ptc.Fp4Matrix(torch.from_numpy(ref.pack(codes, width)).to(DEV), torch.from_numpy(ref.tile(byte)).to(DEV), K,
                      fmt, gt)
    return q, ref.values(codes, byte, K, fmt, g)


def check_product(C, a, b, K, steps=None):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    ulp = ULP[C.dtype]
    tol = (-(-K // 16) + 4) * 2.0 ** -22 * size
    tol = tol + (np.abs(want) + tol) * 2 * ulp + (2.0 ** -24 if C.dtype == torch.float16 else 0.0)
    off = np.abs(host(C) - want)
    assert np.all(off <= tol), f"largest error / bound {np.max(off / np.maximum(tol, 1e-300)):.3g}"


GSHAPES = [(1, 1, 1), (1, 64, 32), (17, 100, 48), (128, 128, 64), (128, 256, 256), (129, 65, 257), (200, 328, 1000),
           (256, 512, 512), (300, 700, 2080), (513, 259, 800)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", GSHAPES)
def test_product(M, N, K, fmt, shape):
    g = (0.37, 1.9) if fmt == "nvfp4" and M % 2 else (None, None)
    A, a = matrix(M, K, fmt, M + N, g=g[0])
    B, b = matrix(N, K, fmt, M + K + 1, g=g[1])
    for dt in DT.values():
        check_product(ptc.matmul_fp4(A, B, out_dtype=dt), a, b, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_of_many_tiles_and_wide_scales(fmt):
    """More tiles than pairs of CTAs (both accumulators in turn), scales over many binades."""
    A, a = matrix(2600, 320, fmt, 1, spread=3.0)
    B, b = matrix(2300, 320, fmt, 2, spread=3.0)
    check_product(ptc.matmul_fp4(A, B, out_dtype=torch.float32), a, b, 320)
    check_product(ptc.matmul_fp4(A, B), a, b, 320)


def test_product_placements(shape):
    """Strided and misaligned outputs, code pitches, another stream; nothing outside C is written."""
    M, N, K = 150, 140, 544
    A, a = matrix(M, K, "mxfp4", 5)
    B, b = matrix(N, K, "mxfp4", 6)
    wide = torch.full((M, 336), 0xFF, dtype=torch.uint8, device=DEV)
    wide[:, :272] = A.codes
    A = ptc.Fp4Matrix(wide[:, :272], A.scales, K)
    for dt in DT.values():
        for off, ld in ((0, 160), (1, 141), (8, 176), (3, 200)):
            buf = torch.full((M * ld + 64,), 7.0, dtype=dt, device=DEV)
            C = buf[off:off + M * ld].view(M, ld)[:, :N]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            ptc.matmul_fp4(A, B, out=C, stream=side)
            side.synchronize()
            check_product(C, a, b, K)
            rest = buf.clone()
            rest[off:off + M * ld].view(M, ld)[:, :N] = 7.0
            assert torch.all(rest == 7.0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_nan_scales_and_garbage_padding(fmt, shape):
    """A NaN block makes its row (column) NaN and no other; scale bytes of rows past the last may hold anything."""
    M, N, K = 140, 70, 320
    A, a = matrix(M, K, fmt, 7)
    B, b = matrix(N, K, fmt, 8)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    kt = A.scales.numel() // 512 // 2
    sa = A.scales.clone()
    for r in range(140, 256):  # padding rows of A
        for t in range(kt):
            o = (r // 128 * kt + t) * 512 + r % 32 * 16 + r % 128 // 32 * 4
            sa[o:o + 4] = nan
    sa[(0 * kt + 1) * 512 + 5 * 16] = nan  # row 5, block 4
    C = host(ptc.matmul_fp4(ptc.Fp4Matrix(A.codes, sa, K, fmt), B, out_dtype=torch.float32))
    assert np.isnan(C[5]).all()
    rows = np.arange(M) != 5
    want = a @ b.T
    assert np.all(np.abs(C - want)[rows] <= ((K / 16 + 4) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T))[rows] + 1e-6 * np.abs(want[rows]))


def test_product_empty_sums_and_sizes():
    A, _ = matrix(5, 32, "mxfp4", 1)
    B, _ = matrix(9, 32, "mxfp4", 2)
    zero = [ptc.Fp4Matrix(m.codes[:, :0], m.scales, 0) for m in (A, B)]
    assert not ptc.matmul_fp4(*zero).any()
    none = ptc.Fp4Matrix(A.codes[:0], A.scales, 32)
    assert ptc.matmul_fp4(none, B).shape == (0, 9) and ptc.matmul_fp4(A, none).shape == (5, 0)


def test_product_is_the_same_every_time(shape):
    A, _ = matrix(260, 1024, "nvfp4", 3)
    B, _ = matrix(300, 1024, "nvfp4", 4)
    first = ptc.matmul_fp4(A, B, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(ptc.matmul_fp4(A, B, out_dtype=torch.float32), first)


@pytest.mark.parametrize("tile", [64, 256])
def test_product_wait_limit_is_reported(tile):
    """Withheld operands: the bounded waits run out, the status is reported, the next call is right."""
    A, a = matrix(300, 512, "mxfp4", 3)
    B, b = matrix(300, 512, "mxfp4", 4)
    ptc.ptc_set_tuning("fp4_tile", tile)
    try:
        ptc.ptc_debug_set_wait_limit(2_000_000, 0)
        ptc.matmul_fp4(A, B)
        torch.cuda.synchronize()
        assert ptc.gemm_poll_device_error() == ptc.PTC_ERR_TIMEOUT
        ptc.ptc_debug_set_wait_limit(0, -1)
        check_product(ptc.matmul_fp4(A, B), a, b, 512)
        assert ptc.gemm_poll_device_error() == ptc.PTC_OK
    finally:
        ptc.ptc_debug_set_wait_limit(0, -1)
        ptc.ptc_set_tuning("fp4_tile", 0)


def test_few_tokens_wait_limit_is_reported():
    """Weights that never arrive: as above for the product of a few tokens."""
    W, w = matrix(300, 1024, "mxfp4", 4)
    x = normal(5, 1024, 1, torch.bfloat16, 0.2)
    try:
        ptc.ptc_debug_set_wait_limit(2_000_000, 0)
        ptc.matmul_a16_fp4(x, W)
        torch.cuda.synchronize()
        assert ptc.gemm_poll_device_error() == ptc.PTC_ERR_TIMEOUT
        ptc.ptc_debug_set_wait_limit(0, -1)
        check_product(ptc.matmul_a16_fp4(x, W), host(x), w, 1024)
        assert ptc.gemm_poll_device_error() == ptc.PTC_OK
    finally:
        ptc.ptc_debug_set_wait_limit(0, -1)


# ------------------------------------------------------------------ few tokens
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 128), (2, 130, 33), (7, 64, 500), (8, 300, 4096), (9, 129, 1000),
                                   (16, 257, 2048), (17, 40, 272), (40, 500, 640), (3, 48, 13000), (16, 200, 9000)])
def test_few_tokens(M, N, K, dtype, fmt):
    W, w = matrix(N, K, fmt, N + K, g=0.5 if fmt == "nvfp4" and M > 3 else None)
    x = normal(M, K, M, DT[dtype], 0.5)
    check_product(ptc.matmul_a16_fp4(x, W), host(x), w, K)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_few_tokens_wide_scales(dtype):
    """mxfp4 scales over the whole exponent range, among them those the one-step expansion cannot reach."""
    N, K = 128, 512
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, size=(N, K))
    byte = np.tile(np.array([90, 127, 143, 160])[:, None], (32, K // 32))
    W = ptc.Fp4Matrix(torch.from_numpy(ref.pack(codes, K // 2)).to(DEV), torch.from_numpy(ref.tile(byte)).to(DEV), K)
    x = (normal(4, K, 1, torch.float32, 0.0) * 1e-9).to(DT[dtype]) if dtype == "bf16" else normal(4, K, 1, DT[dtype], 0.0) * 1e-4
    w = ref.values(codes, byte, K, "mxfp4")
    if dtype == "f16":  # keep the results in binary16's range
        x = (x.float() * 1e-2).to(torch.float16)
    C = host(ptc.matmul_a16_fp4(x, W))
    want, size = host(x) @ w.T, np.abs(host(x)) @ np.abs(w).T
    fits = np.abs(want) < 60000 if dtype == "f16" else np.ones_like(want, dtype=bool)
    tol = (K / 16 + 4) * 2.0 ** -22 * size + np.abs(want) * 2.0 ** (-11 if dtype == "f16" else -8) + 2.0 ** -24 * (dtype == "f16")
    assert fits.sum() > 200 and np.all((np.abs(C - want) <= tol)[fits])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_few_tokens_placements_and_values_that_are_not_finite(fmt):
    W, w = matrix(100, 300, fmt, 3)
    big = normal(6, 700, 4, torch.float16, 0.2)
    for x in (big[:, 1:301], big[::2, 8:308], big[2:3, 5:305]):
        out = torch.full((x.shape[0], 133), 3.0, dtype=torch.float16, device=DEV)
        ptc.matmul_a16_fp4(x, W, out=out[:, 5:105])
        check_product(out[:, 5:105], host(x), w, 300)
        assert torch.all(out[:, :5] == 3) and torch.all(out[:, 105:] == 3)
    for dt in (torch.float16, torch.bfloat16):
        x = normal(3, 300, 5, dt, 0.0)
        x[1, 7] = float("inf")
        x[2, 299] = float("nan")
        C = host(ptc.matmul_a16_fp4(x, W))
        with np.errstate(invalid="ignore"):
            want = host(x) @ w.T
        assert np.isfinite(C[0]).all() and np.isnan(C[2]).all()
        assert np.array_equal(np.isnan(C[1]), np.isnan(want[1])) and np.array_equal(np.isinf(C[1]), np.isinf(want[1]))
    assert ptc.matmul_a16_fp4(x[:0], W).shape == (0, 100)


# ------------------------------------------------------------------ random sizes
@pytest.mark.parametrize("seed", range(24))
def test_random_sizes(seed):
    """Sizes spread over their logarithm, every format and type, by the shapes that the library chooses."""
    rng = np.random.default_rng(100 + seed)

    def size(lo, hi):
        return int(np.exp(rng.uniform(np.log(lo), np.log(hi + 1))))

    fmt = ("mxfp4", "nvfp4")[seed % 2]
    dt = list(DT.values())[seed % 3]
    M, N, K = size(1, 900), size(1, 1500), size(1, 3000)
    A, a = matrix(M, K, fmt, seed)
    B, b = matrix(N, K, fmt, seed + 1, g=0.7 if fmt == "nvfp4" else None)
    check_product(ptc.matmul_fp4(A, B, out_dtype=dt), a, b, K)
    x = normal(size(1, 20), K, seed, (torch.bfloat16, torch.float16)[seed % 4 // 2], 0.5)
    check_product(ptc.matmul_a16_fp4(x, B), host(x), b, K)
    rows, cols = size(1, 600), size(1, 600)
    x = normal(rows, cols, seed, dt)
    bits = ref.bits16(rows, cols, seed, 8, 1)
    xd = ref.dropout(f32(x), 0.15, seed, 8)
    q, t = ptc.quantize_fp4(x, fmt, transposed="both", rounding="stochastic", p=0.15, seed=seed, offset=8)
    check_quantised(q, xd, fmt, "stochastic", bits, None)
    check_quantised(t, np.ascontiguousarray(xd.T), fmt, "stochastic", bits.T, None)


# ------------------------------------------------------------------ offsets past 32 bits
def test_rows_further_apart_than_32_bits_reach():
    """Row pitches that put the last rows more than 2^32 bytes from the first."""
    rows, K = 66000, 64
    A, a = matrix(rows, K, "mxfp4", 1)
    B, b = matrix(48, K, "mxfp4", 2)
    big = torch.empty(rows, 65536 + 64, dtype=torch.uint8, device=DEV)
    codes = big[:, 64:64 + A.codes.shape[1]]
    codes.copy_(A.codes)
    assert codes.stride(0) * (rows - 1) > 2 ** 32
    W = ptc.Fp4Matrix(codes, A.scales, K)
    last = slice(rows - 300, rows)
    out = torch.empty(rows, 32768 + 8, dtype=torch.bfloat16, device=DEV)[:, :48]
    ptc.matmul_fp4(W, B, out=out)
    check_product(out[last], a[last], b, K)
    check_product(out[:300], a[:300], b, K)
    x = normal(3, K, 3, torch.float16, 0.1)
    check_product(ptc.matmul_a16_fp4(x, W)[:, last], host(x), a[last], K)
    v = torch.empty(rows, 32768 + 8, dtype=torch.bfloat16, device=DEV)[:, 3:3 + K]
    ptc.dequantize_fp4(W, out=v)
    assert same(host(v[last]), a[last])
    for q in (ptc.quantize_fp4(v), ptc.quantize_fp4(v, transposed="both")[0]):
        check_quantised(ptc.Fp4Matrix(q.codes[-208:], ptc.Fp4Matrix.tile_scales(q.row_scales()[-208:]), K), f32(v[-208:]),
                        "mxfp4", "nearest", None, None)
    qt = ptc.quantize_fp4(v, transposed=True)
    codes_t, byte_t = ref.quantize(np.ascontiguousarray(f32(v[-208:]).T), "mxfp4")  # 66000 - 208 is a whole block
    assert (rows - 208) % 32 == 0
    got = ref.unpack(qt.codes.cpu().numpy())[:, rows - 208:rows]
    assert np.array_equal(np.where(got == 8, 0, got), np.where(codes_t == 8, 0, codes_t)[:, :208])
    y = ptc.dropout(v, 0.5, 4, 5, out=torch.empty(rows, 32768 + 8, dtype=torch.bfloat16, device=DEV)[:, :K])
    keep = ref.bits16(rows, K, 4, 5, 0)[last] < 32768
    assert same(host(y[last]), np.where(keep, 2 * host(v[last]), 0.0))


# ------------------------------------------------------------------ refusals of the tensor layer
def test_tensor_layer_refusals_on_the_device():
    A, _ = matrix(5, 64, "mxfp4", 1)
    B, _ = matrix(9, 64, "mxfp4", 2)
    x = torch.zeros(5, 64, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, device=DEV)
    wide = torch.zeros(5, 64, 2, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: ptc.matmul_fp4(A, matrix(9, 96, "mxfp4", 2)[0]),           # inner sizes
                lambda: ptc.matmul_fp4(A, matrix(9, 64, "nvfp4", 2)[0]),           # formats
                lambda: ptc.matmul_fp4(A, B, out=torch.zeros(5, 8, device=DEV)),   # out's shape
                lambda: ptc.matmul_fp4(A, B, out=torch.zeros(5, 9)),               # out on the host
                lambda: ptc.matmul_a16_fp4(x[:, :32], B),
                lambda: ptc.matmul_a16_fp4(wide[..., 0], B),                       # column stride 2
                lambda: ptc.matmul_a16_fp4(x, B, out=torch.zeros(5, 9, device=DEV)),
                lambda: ptc.dropout(x, 0.1, 1, residual=x[:4]),
                lambda: ptc.dropout(x, 0.1, 1, out=torch.zeros(5, 64, device=DEV)),
                lambda: ptc.dropout(x[:1].expand(5, 64), 0.1, 1),                  # rows that overlap
                lambda: ptc.dropout(x.view(-1), 0.1, 1),
                lambda: ptc.quantize_fp4(x, "fp4"),
                lambda: ptc.quantize_fp4(x, tensor_scale=one),                     # mxfp4 has none
                lambda: ptc.quantize_fp4(x, "nvfp4", tensor_scale=torch.ones(1)),
                lambda: ptc.quantize_fp4(x, "nvfp4", tensor_scale=one.double()),
                lambda: ptc.dequantize_fp4(A, out=torch.zeros(5, 63, device=DEV)),
                lambda: ptc.Fp4Matrix(A.codes, A.scales[:-1], 64),
                lambda: ptc.Fp4Matrix(A.codes[:, :16], A.scales, 64),
                lambda: ptc.Fp4Matrix(A.codes, A.scales, -1),
                lambda: ptc.Fp4Matrix(torch.zeros(5, 40, dtype=torch.uint8, device=DEV), A.scales, 64)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ptc.matmul_fp4(A, x), lambda: ptc.matmul_fp4(A, B, out_dtype=torch.float64),
                lambda: ptc.matmul_a16_fp4(x.float(), B), lambda: ptc.quantize_fp4(x.int()), lambda: ptc.dropout(3, 0.1, 1),
                lambda: ptc.Fp4Matrix(A.codes.int(), A.scales, 64), lambda: ptc.matmul_fp4(A, B, out_dtype="bf16")):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ptc.dropout(x, 1.5, 1), lambda: ptc.dropout(x, 0.1, 1, offset=-1),
                lambda: ptc.dropout(x[:, :60], 0.1, 1, out=x[:, 4:])):
        with pytest.raises(ptc.PtcError):
            bad()
    none = ptc.quantize_fp4(x[:, :0])
    assert none.shape == (5, 0) and not ptc.matmul_fp4(none, ptc.quantize_fp4(x[:3, :0])).any()
    assert not ptc.matmul_a16_fp4(x[:, :0], none).any() and ptc.dequantize_fp4(none).shape == (5, 0)
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("tokens,inputs,outputs,p", [(1, 32, 16, 0.0), (65, 200, 130, 0.25), (256, 512, 384, 0.1)])
def test_linear_step(tokens, inputs, outputs, p):
    x = normal(tokens, inputs, 1, torch.bfloat16, 0.3)
    w = normal(outputs, inputs, 2, torch.bfloat16, 0.1)
    dy = normal(tokens, outputs, 3, torch.bfloat16, 0.1)
    y, saved = fp4_linear.forward(x, w, p=p, seed=SEED, offset=6)
    dx, dw = fp4_linear.backward(dy, saved)

    def q(v, rounding="nearest", bits=None):
        v = np.ascontiguousarray(v)
        return ref.values(*ref.quantize(v, "mxfp4", rounding, bits), v.shape[1], "mxfp4")

    xd = ref.dropout(f32(x), p, SEED, 6) if p else f32(x)
    bits = ref.bits16(tokens, outputs, SEED, 6, 1)
    dq, dqt = q(f32(dy), "stochastic", bits), q(f32(dy).T, "stochastic", bits.T)
    check_product(y, q(xd), q(f32(w)), inputs)
    check_product(dw, dqt, q(xd.T), tokens)
    a, b = dq, q(f32(w).T)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (outputs / 16 + 4) * 2.0 ** -22 * size + np.abs(want) * 2.0 ** -7
    if p:
        keep = ref.bits16(tokens, inputs, SEED, 6, 0) < int((1 - p) * 65536 + 0.5)
        scale = 65536 / int((1 - p) * 65536 + 0.5)
        want, tol = np.where(keep, want * scale, 0.0), np.where(keep, tol * scale, 0.0)
    assert np.all(np.abs(host(dx) - want) <= tol)


def test_linear_gradients_by_differences():
    """Operands that the format holds exactly make the layer linear in each of them: differences of
    L = sum(dy * y) are exact and equal the gradients."""
    rng = np.random.default_rng(4)
    vals = np.array([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], dtype=np.float32)

    def pick(*s):
        v = rng.choice(vals, size=s).astype(np.float32)
        v[:, ::32] = 6.0  # every block along the rows ...
        v[::32, :] = 6.0  # ... and along the columns has scale 1
        return torch.from_numpy(v).to(DEV)

    x, w, dy = pick(64, 96), pick(32, 96), pick(64, 32)
    y, saved = fp4_linear.forward(x, w)
    dx, dw = fp4_linear.backward(dy, saved)
    assert torch.equal(y, x @ w.t()) and torch.equal(dx, dy @ w) and torch.equal(dw, dy.t() @ x)
    loss = float((dy.double() * y.double()).sum())
    for i, j in [(1, 1), (33, 40), (63, 95)]:
        for t, grad, fw in ((x, dx, lambda v: fp4_linear.forward(v, w)[0]), (w, dw, lambda v: fp4_linear.forward(x, v)[0])):
            i2 = i % t.shape[0]
            v = t.clone()
            step = -1.0 if v[i2, j] == 1 else 1.0 - float(v[i2, j])  # to 1 (or 0): held exactly too
            v[i2, j] += step
            diff = (float((dy.double() * fw(v).double()).sum()) - loss) / step
            assert diff == float(grad[i2, j])


def test_operators_in_a_cuda_graph():
    x = normal(64, 256, 1, torch.bfloat16, 0.3)
    w = normal(128, 256, 2, torch.bfloat16, 0.1)
    dy = normal(64, 128, 3, torch.bfloat16, 0.1)
    step = lambda: (lambda y, s: (y, *fp4_linear.backward(dy, s)))(*fp4_linear.forward(x, w, 0.1, 3, 4))  # noqa: E731
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
