"""Without a GPU: the 4-bit reference against published and independent values,
and what the 4-bit entry points refuse (before any CUDA call; the addresses
passed here are never dereferenced)."""
import numpy as np
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests import fp4_ref as ref

BASE = 1 << 40
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return ptc.lib()


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_published_vectors(ctr, key, want):
    """The known-answer vectors published with the generator."""
    assert tuple(int(v) for v in ref.philox(np.array(ctr, dtype=np.uint64), key)) == want


def test_e4m3_against_torch():
    b = torch.arange(0x7F, dtype=torch.uint8)
    assert np.array_equal(b.view(torch.float8_e4m3fn).double().numpy(), ref.E4M3)
    v = torch.cat([torch.rand(4000) * 448, torch.rand(2000) * 2.0 ** -7, torch.from_numpy((ref.E4M3[1:] + ref.E4M3[:-1]) / 2).float()])
    assert np.array_equal(v.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), ref.e4m3_nearest(v.numpy()))


def test_reference_quantisation_is_the_nearest_value():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 96)) * np.exp2(rng.integers(-20, 20, (40, 1)))).astype(np.float32)
    codes, byte = ref.quantize(x, "mxfp4")
    s = np.repeat(ref.scale_value(byte, "mxfp4"), 32, axis=1)
    grid = np.concatenate([-ref.GRID[:0:-1], ref.GRID])
    near = grid[np.abs(x[..., None] / s[..., None] - grid).argmin(-1)] * s
    got = ref.values(codes, byte, 96, "mxfp4")
    assert np.array_equal(np.abs(got - x), np.abs(near - x))
    v = ref.unpack(ref.pack(codes, 64))
    assert np.array_equal(v[:, :96], codes) and not v[:, 96:].any()


def test_reference_quantisation_keeps_ties_to_even():
    """Midpoints of the grid times every E4M3 scale round to the even code."""
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    even = np.array([0, 1, 1, 2, 2, 4, 4])
    d = ref.E4M3[8:].astype(np.float32)[:, None]
    x = np.concatenate([6 * d, mid * d, np.zeros((d.shape[0], 8), np.float32)], axis=1)
    codes, byte = ref.quantize(x, "nvfp4")
    assert np.array_equal(ref.E4M3[byte[:, 0]], d[:, 0]) and np.all(ref.GRID[codes[:, 1:8]] == even)


def test_tiles_round_trip():
    byte = torch.from_numpy(np.random.default_rng(1).integers(0, 255, (200, 9)).astype(np.uint8))
    t = ptc.Fp4Matrix.tile_scales(byte)
    assert np.array_equal(t.numpy(), ref.tile(byte.numpy()))
    assert t.numel() == ptc.fp4_scale_bytes(200, 9 * 32, "mxfp4") == ptc.fp4_scale_bytes(200, 9 * 16, "nvfp4")


GEMM = dict(M=64, N=96, K=100, fmt=0, A=BASE, lda=64, SA=BASE + GB, GA=None, B=BASE + 2 * GB, ldb=80, SB=BASE + 3 * GB,
            GB=None, C=BASE + 4 * GB, ldc=96, out=1)


def gemm(L, **kw):
    a = {**GEMM, **kw}
    return L.gemm_fp4(a["M"], a["N"], a["K"], a["fmt"], a["A"], a["lda"], a["SA"], a["GA"], a["B"], a["ldb"], a["SB"],
                      a["GB"], a["C"], a["ldc"], a["out"], None)


def test_gemm_fp4_refusals(L):
    for bad in (dict(M=-1), dict(N=GB + 1), dict(K=-3), dict(M=GB, N=GB), dict(fmt=2), dict(out=3), dict(A=None),
                dict(SB=None), dict(C=None), dict(lda=48), dict(ldb=0), dict(ldc=95), dict(ldc=(1 << 36) + 1),
                dict(lda=(1 << 36) + 16), dict(GA=BASE + 5 * GB)):
        assert gemm(L, **bad) == ptc.PTC_ERR_INVALID, bad
    for bad in (dict(A=BASE + 8), dict(SB=BASE + 3 * GB + 4), dict(lda=72), dict(C=BASE + 4 * GB + 1),
                dict(out=0, C=BASE + 4 * GB + 2), dict(fmt=1, GB=BASE + 5 * GB + 2)):
        assert gemm(L, **bad) == ptc.PTC_ERR_ALIGN, bad
    for bad in (dict(C=BASE), dict(C=BASE + 63 * 64 + 62), dict(C=BASE + GB + 510), dict(C=BASE + 2 * GB - 2),
                dict(fmt=1, GA=BASE + 4 * GB + 64)):
        assert gemm(L, **bad) == ptc.PTC_ERR_OVERLAP, bad
    assert gemm(L, M=0, A=None, C=None) == ptc.PTC_OK and gemm(L, N=0, B=None, C=None) == ptc.PTC_OK


def test_gemm_a16_fp4_refusals(L):
    good = dict(M=3, N=96, K=100, type=1, X=BASE, ldx=100, fmt=0, W=BASE + GB, ldw=64, SW=BASE + 2 * GB, GW=None,
                C=BASE + 3 * GB, ldc=96)

    def call(**kw):
        a = {**good, **kw}
        return L.gemm_a16_fp4(a["M"], a["N"], a["K"], a["type"], a["X"], a["ldx"], a["fmt"], a["W"], a["ldw"], a["SW"],
                              a["GW"], a["C"], a["ldc"], None)

    for bad in (dict(M=-1), dict(K=GB + 1), dict(M=1 << 20), dict(type=0), dict(type=5), dict(fmt=-1), dict(X=None),
                dict(W=None), dict(C=None), dict(ldx=99), dict(ldc=95), dict(ldw=48), dict(GW=BASE + 5 * GB)):
        assert call(**bad) == ptc.PTC_ERR_INVALID, bad
    for bad in (dict(X=BASE + 1), dict(W=BASE + GB + 8), dict(SW=BASE + 2 * GB + 1), dict(ldw=72), dict(C=BASE + 3 * GB + 1)):
        assert call(**bad) == ptc.PTC_ERR_ALIGN, bad
    for bad in (dict(C=BASE + 2), dict(C=BASE + GB + 64), dict(C=BASE + 2 * GB + 2)):
        assert call(**bad) == ptc.PTC_ERR_OVERLAP, bad
    assert call(M=0, X=None, C=None) == ptc.PTC_OK


def test_dropout_refusals(L):
    def call(rows=4, cols=100, x=BASE, ldx=100, r=None, ldr=0, y=BASE + GB, ldy=100, type=1, p=0.5, seed=1, offset=0):
        return L.ptc_dropout(rows, cols, x, ldx, r, ldr, y, ldy, type, p, seed, offset, None)

    for bad in (dict(rows=-1), dict(cols=GB + 1), dict(type=3), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")),
                dict(offset=1 << 63), dict(x=None), dict(y=None), dict(ldx=99), dict(ldy=50), dict(r=BASE + 2 * GB, ldr=3)):
        assert call(**bad) == ptc.PTC_ERR_INVALID, bad
    for bad in (dict(x=BASE + 1), dict(y=BASE + GB + 2, type=0), dict(r=BASE + 2 * GB + 1, ldr=100)):
        assert call(**bad) == ptc.PTC_ERR_ALIGN, bad
    for bad in (dict(y=BASE + 2), dict(y=BASE, ldy=104), dict(r=BASE + GB + 8, ldr=100)):
        assert call(**bad) == ptc.PTC_ERR_OVERLAP, bad
    assert call(rows=0, x=None, y=None) == ptc.PTC_OK


def test_quantize_fp4_refusals(L):
    good = dict(rows=40, cols=100, x=BASE, ldx=100, type=1, fmt=0, rounding=0, g=None, c=BASE + GB, pitch=64,
                s=BASE + 2 * GB, ct=None, pt=0, st=None, p=0.0, seed=0, offset=0)

    def call(**kw):
        a = {**good, **kw}
        return L.ptc_quantize_fp4(a["rows"], a["cols"], a["x"], a["ldx"], a["type"], a["fmt"], a["rounding"], a["g"], a["c"],
                                  a["pitch"], a["s"], a["ct"], a["pt"], a["st"], a["p"], a["seed"], a["offset"], None)

    both = dict(ct=BASE + 3 * GB, pt=32, st=BASE + 4 * GB)
    for bad in (dict(rows=-1), dict(type=9), dict(fmt=2), dict(rounding=2), dict(p=2.0), dict(offset=1 << 63), dict(x=None),
                dict(c=None), dict(s=None), dict(ldx=99), dict(pitch=48), dict(g=BASE + 5 * GB), {**both, "pt": 16},
                {**both, "st": None}):
        assert call(**bad) == ptc.PTC_ERR_INVALID, bad
    for bad in (dict(x=BASE + 1), dict(c=BASE + GB + 4), dict(pitch=72), dict(s=BASE + 2 * GB + 8),
                dict(fmt=1, g=BASE + 5 * GB + 1), {**both, "ct": BASE + 3 * GB + 2}):
        assert call(**bad) == ptc.PTC_ERR_ALIGN, bad
    for bad in (dict(c=BASE), dict(s=BASE + GB + 64), {**both, "st": BASE + 2 * GB}, {**both, "ct": BASE + 16},
                dict(fmt=1, g=BASE + GB)):
        assert call(**bad) == ptc.PTC_ERR_OVERLAP, bad
    assert call(rows=0, x=None) == ptc.PTC_OK


def test_dequantize_fp4_refusals(L):
    def call(rows=4, cols=100, c=BASE, pitch=64, s=BASE + GB, fmt=0, g=None, y=BASE + 2 * GB, ldy=100, type=0):
        return L.ptc_dequantize_fp4(rows, cols, c, pitch, s, fmt, g, y, ldy, type, None)

    for bad in (dict(rows=-1), dict(type=3), dict(fmt=3), dict(c=None), dict(s=None), dict(y=None), dict(pitch=32),
                dict(ldy=99), dict(g=BASE + 3 * GB)):
        assert call(**bad) == ptc.PTC_ERR_INVALID, bad
    for bad in (dict(c=BASE + 1), dict(pitch=65), dict(s=BASE + GB + 2), dict(y=BASE + 2 * GB + 2)):
        assert call(**bad) == ptc.PTC_ERR_ALIGN, bad
    for bad in (dict(y=BASE + 16), dict(y=BASE + GB + 4)):
        assert call(**bad) == ptc.PTC_ERR_OVERLAP, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path only")
def test_no_device_is_reported(L):
    assert gemm(L) == ptc.PTC_ERR_DEVICE
    assert L.ptc_dropout(4, 8, BASE, 8, None, 0, BASE + GB, 8, 1, 0.5, 1, 0, None) == ptc.PTC_ERR_DEVICE


def test_tuning_keys(L):
    for key, bad, good in (("fp4_tile", 32, 0), ("fp4_tile", 192, 0), ("fp4_ksplit", 3, 0), ("fp4_ksplit", 16, 0),
                           ("fp4_group_m", 0, 8)):
        with pytest.raises(ptc.PtcError):
            ptc.ptc_set_tuning(key, bad)
        assert ptc.ptc_set_tuning(key, good) == 0


def test_tensor_layer_refusals(L):
    codes, scales = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # host tensors
        ptc.dropout(x, 0.5, 1)
    with pytest.raises(ValueError):
        ptc.quantize_fp4(x)
    with pytest.raises(ValueError):
        ptc.Fp4Matrix(codes, scales, 32)
    with pytest.raises(ValueError):
        ptc.Fp4Matrix(codes, scales, 32, "fp4")
    with pytest.raises(TypeError):
        ptc.Fp4Matrix(codes.int(), scales, 32)
    with pytest.raises(TypeError):
        ptc.dropout(x.double(), 0.5, 1)
    for kw in (dict(fmt="e2m1"), dict(rounding="up"), dict(transposed="only")):
        with pytest.raises(ValueError):
            ptc.quantize_fp4(x, **kw)
    with pytest.raises(TypeError):
        ptc.matmul_a16_fp4(x.float(), None)
