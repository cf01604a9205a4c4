"""Dropout, quantisation and its inverse at sizes where the kernels take several
column groups per row, four loads per lane and more than one step per thread.

Functions of their inputs to the last bit: compared for equality with the plain
reference on rows (and columns) from the start, the middle and the end."""
import numpy as np
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests import fp4_ref as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
SEED, OFFSET = 0x123456789ABCDEF1, (3 << 33) + 5
# (rows, columns, elements by which rows are further apart): rows aligned to 16 bytes and not, remainders of every group size
SIZES = [(10000, 1000, 0), (5000, 2090, 0), (9000, 1032, 0), (20011, 520, 8), (9731, 1024, 0), (3300, 4099, 5)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def data(rows, cols, pad, dtype):
    g = torch.Generator(DEV).manual_seed(rows)
    x = torch.randn(rows, cols + pad, generator=g, device=DEV) * torch.exp(2 * torch.randn(1, cols + pad, generator=g, device=DEV))
    return x.to(dtype)[:, :cols]


def some(n, count=70):
    """Indexes from the start, the middle and the end, the last in whole."""
    return np.unique(np.concatenate([np.arange(min(n, count)), n // 2 + np.arange(min(n - n // 2, count)), np.arange(max(0, n - 200), n)]))


def bits(rows, cols, purpose):
    """The 16 random bits of the elements at these rows and columns."""
    ctr = np.zeros((len(rows), len(cols), 4), dtype=np.uint64)
    ctr[..., 0], ctr[..., 1] = cols // 8, rows[:, None]
    ctr[..., 2], ctr[..., 3] = OFFSET & 0xFFFFFFFF, (OFFSET >> 32) | (purpose << 31)
    w = ref.philox(ctr, (SEED & 0xFFFFFFFF, SEED >> 32))
    word = np.take_along_axis(w, np.broadcast_to((cols % 8 // 2)[:, None], w.shape[:2] + (1,)), -1)[..., 0]
    return (word >> (16 * (cols % 2)).astype(np.uint64) & np.uint64(0xFFFF)).astype(np.int64)


def dropped(x, rows, cols, p):
    """FP32 values after dropout of x's elements there."""
    if p == 0:
        return x
    kept = int((1 - p) * 65536 + 0.5)
    return np.where(bits(rows, cols, 0) < kept, x * np.float32(65536 / kept), np.float32(0))


def compare(q, which, x, fmt, rounding, b, g):
    """Rows `which` of q against the reference of their values x."""
    codes, byte = ref.quantize(x, fmt, rounding, b, g)
    width = 16 * -(-x.shape[1] // 32)
    at = torch.from_numpy(which).to(DEV)
    got = ref.unpack(q.codes[at].cpu().numpy())
    assert q.codes.shape[1] == width
    assert np.array_equal(np.where(got == 8, 0, got), ref.unpack(ref.pack(codes, width)))
    assert np.array_equal(q.row_scales()[at].cpu().numpy(), byte)
    return codes, byte


def padding_is_zero(q, fmt):
    """Scale bytes of rows past the last and of blocks past K."""
    rows, K = q.shape
    blocks = -(-K // ref.BLOCK[fmt])
    kt = -(-blocks // 4)
    s = q.scales.view(-1, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kt * 4)
    assert not s[rows:].any() and not s[:, blocks:].any()


@pytest.mark.parametrize("rounding,p", [("nearest", 0.0), ("stochastic", 0.0), ("nearest", 0.2), ("stochastic", 0.2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,pad", SIZES)
def test_quantize(rows, cols, pad, fmt, dtype, rounding, p):
    x = data(rows, cols, pad, dtype)
    g = (x.float().abs().amax() / 2000).reshape(1) if fmt == "nvfp4" else None
    gv = None if g is None else np.float32(g.item())
    kw = dict(rounding=rounding, tensor_scale=g, p=p, seed=SEED, offset=OFFSET)
    r, c = some(rows), some(cols, 20)[::3]
    all_r, all_c = np.arange(rows), np.arange(cols)
    xr = dropped(x[torch.from_numpy(r).to(DEV)].cpu().float().numpy(), r, all_c, p)
    xc = dropped(x[:, torch.from_numpy(c).to(DEV)].cpu().float().numpy(), all_r, c, p)
    br, bc = (bits(r, all_c, 1), bits(all_r, c, 1).T) if rounding == "stochastic" else (None, None)
    one = ptc.quantize_fp4(x, fmt, **kw)
    codes, byte = compare(one, r, xr, fmt, rounding, br, gv)
    both, t = ptc.quantize_fp4(x, fmt, transposed="both", **kw)
    assert torch.equal(both.codes, one.codes) and torch.equal(both.scales, one.scales)
    compare(t, c, np.ascontiguousarray(xc.T), fmt, rounding, bc, gv)
    only = ptc.quantize_fp4(x, fmt, transposed=True, **kw)
    assert torch.equal(only.codes, t.codes) and torch.equal(only.scales, t.scales)
    padding_is_zero(one, fmt)
    padding_is_zero(t, fmt)
    # and back, to rows aligned and not
    v = ref.values(codes, byte, cols, fmt).astype(np.float32)
    v = v if gv is None else v * gv
    at = torch.from_numpy(r).to(DEV)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        want = torch.from_numpy(v).to(dt)
        assert torch.equal(ptc.dequantize_fp4(one, dt)[at].cpu(), want)
        wide = torch.full((rows, cols + 3), 9.0, dtype=dt, device=DEV)
        ptc.dequantize_fp4(one, out=wide[:, 1:cols + 1])
        assert torch.equal(wide[at, 1:cols + 1].cpu(), want)
        assert bool((wide[:, 0] == 9).all()) and bool((wide[:, cols + 1:] == 9).all())


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,cols,pad", SIZES + [(700000, 9, 0), (650000, 8, 0)])
def test_dropout(rows, cols, pad, dtype, residual):
    x = data(rows, cols, pad, dtype)
    res = data(rows + 1, cols, pad, dtype)[1:] if residual else None
    y = ptc.dropout(x, 0.2, SEED, OFFSET, residual=res)
    r = some(rows)
    at = torch.from_numpy(r).to(DEV)
    want = dropped(x[at].cpu().float().numpy(), r, np.arange(cols), 0.2)
    if residual:
        want = want + res[at].cpu().float().numpy()
    assert torch.equal(y[at].cpu(), torch.from_numpy(want.astype(np.float32)).to(dtype))
    kept = (y != 0).float().mean().item() if not residual else 0.8
    assert abs(kept - 0.8) < 0.002
    if dtype == torch.float32 and not residual:
        half = ptc.dropout(x, 0.2, SEED, OFFSET, out_dtype=torch.bfloat16)
        assert torch.equal(half, y.bfloat16())
