"""Plain 64-bit reference of the counter-based generator and of the microscaled
4-bit formats (numpy, on the host), written from the definitions in
include/ptc.h.  Where a definition rounds to FP32, the step is done in
np.float32; everything else is float64."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def philox(ctr, key):
    """Philox4x32-10 of counters (..., 4) and a 64-bit key given as (low, high)."""
    c = [np.asarray(ctr[..., i], dtype=np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1),
             p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=-1)


def bits16(rows, cols, seed, offset, purpose):
    groups = (cols + 7) // 8
    ctr = np.zeros((rows, groups, 4), dtype=np.uint64)
    ctr[..., 0] = np.arange(groups)
    ctr[..., 1] = np.arange(rows)[:, None]
    ctr[..., 2] = offset & 0xFFFFFFFF
    ctr[..., 3] = (offset >> 32) | (purpose << 31)
    w = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    out = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=-1).reshape(rows, groups * 8)
    return out[:, :cols].astype(np.int64)


def dropout(x, p, seed, offset, residual=None):
    """FP32 result of x (any float array, exact in FP32) before the output rounding."""
    kept = int(np.floor((1 - p) * 65536 + 0.5))
    scale = np.float32(65536 / max(kept, 1))
    keep = bits16(*x.shape, seed, offset, 0) < kept
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.where(keep, x.astype(np.float32) * scale, np.float32(0))
        return y if residual is None else (y + residual.astype(np.float32))


def e4m3_value(byte):
    b = np.asarray(byte).astype(np.int64) & 0x7F
    e, m = b >> 3, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b == 0x7F, np.nan, v)


E4M3 = e4m3_value(np.arange(0x7F))


def e4m3_nearest(v):
    """Byte of the nearest non-negative E4M3 number, ties to the even byte, at most 448."""
    v = np.minimum(np.asarray(v, dtype=np.float64), 448.0)
    at = np.searchsorted(E4M3, v, side="right") - 1
    up = np.minimum(at + 1, 0x7E)
    d0, d1 = v - E4M3[at], E4M3[up] - v
    return np.where((d1 < d0) | ((d1 == d0) & (at % 2 == 1)), up, at)


def scale_value(byte, fmt):
    b = np.asarray(byte)
    if fmt == "nvfp4":
        return e4m3_value(b)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 127))


def quantize(x, fmt, rounding="nearest", bits=None, g=None):
    """(codes, one per entry, rows padded to whole blocks; scale bytes (rows, blocks))."""
    n = BLOCK[fmt]
    rows, cols = x.shape
    blocks = -(-cols // n)
    full = np.zeros((rows, blocks * n), dtype=np.float32)
    full[:, :cols] = x
    r = np.zeros((rows, blocks * n), dtype=np.int64)
    if bits is not None:
        r[:, :cols] = bits
    full, r = full.reshape(rows, blocks, n), r.reshape(rows, blocks, n)
    finite = np.isfinite(full).all(-1)
    v = np.where(finite[..., None], full, np.float32(0))
    a = np.abs(v).max(-1)
    if fmt == "mxfp4":
        m, e = np.frexp(a.astype(np.float64))  # a = m 2^e, 1/2 <= m < 1
        e = e.astype(np.int64) - 1 - 2
        if rounding == "stochastic":
            e = e + (m > 0.75)
        byte = np.where(a > 0, np.clip(e + 127, 0, 254), 0)
        d = np.ldexp(np.float64(1), byte - 127)
    else:
        gs = np.float32(1 if g is None else g)
        six = np.float32(gs * np.float32(6))
        with np.errstate(over="ignore"):
            byte = e4m3_nearest((a / six).astype(np.float32))
        if rounding == "stochastic":
            byte = np.where((six * E4M3[byte].astype(np.float32) < a) & (byte < 0x7E), byte + 1, byte)
        d = E4M3[byte].astype(np.float32) * gs
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        # the quotient rounded to FP32, as the definition has it (mxfp4: exact)
        u = np.where(d[..., None] > 0, np.abs(v) / d[..., None].astype(np.float64), 0.0).astype(np.float32)
    u = np.minimum(u.astype(np.float64), 6.0)
    low = np.minimum(np.searchsorted(GRID, u, side="right") - 1, 7)
    high = np.minimum(low + 1, 7)
    if rounding == "nearest":
        mid = (GRID[low] + GRID[high]) / 2
        up = (u > mid) | ((u == mid) & (low % 2 == 1))
    else:
        gap = np.where(high > low, GRID[high] - GRID[low], 1.0)
        up = (u - GRID[low]) / gap >= 1 - r / 65536
    code = np.where(up, high, low)
    code = code + 8 * ((v < 0) & (code > 0))
    nan = 0x7F if fmt == "nvfp4" else 255
    return np.where(finite[..., None], code, 0).reshape(rows, -1), np.where(finite, byte, nan)


def values(codes, byte, cols, fmt, g=None):
    """float64 values of codes (one per entry) and scale bytes."""
    n = BLOCK[fmt]
    rows, blocks = byte.shape
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    v = v[:, :blocks * n].reshape(rows, blocks, n) * scale_value(byte, fmt)[..., None]
    return v.reshape(rows, -1)[:, :cols] * (1.0 if g is None else float(g))


def pack(codes, width):
    """Two codes per byte, low nibble first, rows of `width` bytes."""
    out = np.zeros((codes.shape[0], width), dtype=np.uint8)
    c = np.zeros((codes.shape[0], 2 * width), dtype=np.uint8)
    c[:, :codes.shape[1]] = codes
    out[:] = c[:, 0::2] | (c[:, 1::2] << 4)
    return out


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(packed.shape[0], -1).astype(np.int64)


def tile(byte):
    """Row-major scale bytes to tiles of 128 rows x 4 blocks, one by one."""
    rows, blocks = byte.shape
    kt = -(-blocks // 4)
    out = np.zeros(-(-rows // 128) * kt * 512, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    out[(r // 128 * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = byte
    return out
