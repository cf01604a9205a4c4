"""Performance cases of the 4-bit operators: counter-based dropout, microscaled
4-bit quantisation, the product of two 4-bit matrices, the product of 16-bit
activations with 4-bit weights, and one training step of a linear layer that
uses them together.

Each case is computed either in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, by the calls a
user makes of the library.  ``exact`` gives the same outputs from the
operators' definitions in 64 bits.

Formats.  A microscaled matrix holds 4-bit codes (sign, two exponent bits, one
mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two per byte with the even element
in the low nibble, and one scale byte per block of consecutive elements of a
row: a power of two (exponent byte, bias 127) per 32 elements ("mxfp4"), or an
E4M3 number per 16 elements and one FP32 scale for the matrix ("nvfp4").  Code
rows are padded with zeros to 16 bytes; scale bytes are stored in tiles of 128
rows x 4 blocks (512 bytes: byte (r % 32) * 16 + (r / 32) * 4 + block % 4 of a
tile, the tiles of 128 rows in order of the block), padded with zeros.

Random numbers.  16 bits per element from Philox4x32-10 (Salmon et al.,
"Parallel random numbers: as easy as 1, 2, 3", SC 2011): counter (column / 8,
row, offset low, offset high | purpose << 31), key = seed; element column % 8
takes bits 16 * (column % 2) of word (column % 8) / 2.
"""
import math

import numpy as np
import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token's activations before a 4-bit product: latency counts
        dict(name="quantise one token", op="quantise", rows=1, cols=4096, fmt="mxfp4", dtype="bf16",
             transposed="no", rounding="nearest", p=0.0),
        # the activations of a long prompt or a training batch
        dict(name="quantise a batch", op="quantise", rows=8192, cols=8192, fmt="mxfp4", dtype="bf16",
             transposed="no", rounding="nearest", p=0.0),
        # a gradient of odd sizes, for both gradient products at once, without bias
        dict(name="quantise a gradient both ways", op="quantise", rows=2047, cols=1003, fmt="nvfp4", dtype="f16",
             transposed="both", rounding="stochastic", p=0.1),
        # dropout of a block's output, added to the residual stream
        dict(name="dropout with residual", op="dropout", rows=8192, cols=8192, dtype="bf16", p=0.1, residual=True),
        # the backward pass of a small FP32 layer with odd sizes
        dict(name="dropout of a small gradient", op="dropout", rows=333, cols=777, dtype="f32", p=0.5,
             residual=False),
        # the smallest square product of the benchmark's sizes
        dict(name="product 512", op="product", m=512, n=512, k=512, fmt="mxfp4", out="bf16"),
        # the middle of the benchmark's sizes: one wave of tiles
        dict(name="product 2048", op="product", m=2048, n=2048, k=2048, fmt="nvfp4", out="f16"),
        # the benchmark's largest size
        dict(name="product 8192", op="product", m=8192, n=8192, k=8192, fmt="mxfp4", out="bf16"),
        # a ragged prompt against a layer of uneven sizes, FP32 logits
        dict(name="product ragged", op="product", m=1001, n=1339, k=2090, fmt="nvfp4", out="f32"),
        # decoding one sequence: the weights are read once
        dict(name="one token, 4-bit weights", op="tokens", m=1, n=4096, k=4096, fmt="mxfp4", dtype="bf16"),
        # decoding a batch of sequences against a wide layer
        dict(name="sixteen tokens, 4-bit weights", op="tokens", m=16, n=16384, k=8192, fmt="nvfp4", dtype="f16"),
        # forward and backward of a linear layer with dropout of its input
        dict(name="training step", op="step", tokens=4096, inputs=2048, outputs=8192, dtype="bf16", p=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantise", "quantise", "dropout", "dropout", "product", "product", "product", "tokens",
                     "tokens", "step"])
    if op == "quantise":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 16, 8192), fmt=rng.choice(["mxfp4", "nvfp4"]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), transposed=rng.choice(["no", "only", "both"]),
                    rounding=rng.choice(["nearest", "stochastic"]), p=rng.choice([0.0, 0.0, 0.1, 0.25]))
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 1, 8192),
                    dtype=rng.choice(["bf16", "f16", "f32"]), p=rng.choice([0.1, 0.2, 0.5]),
                    residual=rng.choice([True, False]))
    if op == "product":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 16, 8192), k=_log(rng, 32, 8192),
                    fmt=rng.choice(["mxfp4", "nvfp4"]), out=rng.choice(["bf16", "f16", "f32"]))
    if op == "tokens":
        return dict(op=op, m=rng.randint(1, 16), n=_log(rng, 64, 16384), k=_log(rng, 64, 8192),
                    fmt=rng.choice(["mxfp4", "nvfp4"]), dtype=rng.choice(["bf16", "f16"]))
    return dict(op=op, tokens=_log(rng, 32, 4096), inputs=_log(rng, 64, 2048), outputs=_log(rng, 64, 8192),
                dtype=rng.choice(["bf16", "f16"]), p=rng.choice([0.0, 0.1, 0.3]))


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}

    def held(rows, cols, fmt):  # codes and scales
        return rows * cols / 2 + rows * math.ceil(cols / BLOCK[fmt])

    if op == "quantise":
        r, k, out = c["rows"], c["cols"], 0
        if c["transposed"] != "only":
            out += held(r, k, c["fmt"]) + 2 * r * k
        if c["transposed"] != "no":
            out += held(k, r, c["fmt"]) + 2 * r * k
        return dict(bytes=r * k * size[c["dtype"]] + out, flops=4 * r * k)
    if op == "dropout":
        return dict(bytes=c["rows"] * c["cols"] * size[c["dtype"]] * (3 if c["residual"] else 2),
                    flops=2 * c["rows"] * c["cols"])
    if op == "product":
        return dict(bytes=held(c["m"], c["k"], c["fmt"]) + held(c["n"], c["k"], c["fmt"])
                    + c["m"] * c["n"] * size[c["out"]], flops=2 * c["m"] * c["n"] * c["k"])
    if op == "tokens":
        return dict(bytes=held(c["n"], c["k"], c["fmt"]) + 2 * c["m"] * (c["n"] + c["k"]),
                    flops=2 * c["m"] * c["n"] * c["k"])
    t, i, o = c["tokens"], c["inputs"], c["outputs"]
    # x, w, dy read; y, dx (16 bits) and dw (32 bits) written; three products
    return dict(bytes=2 * (t * i + o * i + t * o) + 2 * (t * o + t * i) + 4 * o * i, flops=6 * t * i * o)


# ------------------------------------------------------------------ inputs
def _normal(g, rows, cols, dtype):
    """Activations: normal values with a spread of channel sizes and a few large channels."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    size = torch.exp(0.7 * torch.randn((1, cols), generator=g, device="cuda"))
    size = torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.01, size * 10, size)
    return (x * size).to(dtype)


def _scale_of(x):
    """The matrix scale of "nvfp4": the largest value becomes 448 * 6."""
    return (x.abs().amax().float() / 2688.0).reshape(1)


def _held(g, rows, cols, fmt):
    x = torch.randn((rows, cols), generator=g, device="cuda") / math.sqrt(cols)
    gs = _scale_of(x) if fmt == "nvfp4" else None
    codes, scales = _quantise(x, fmt, "nearest", None, gs)
    return _pack(codes), _tile(scales), gs


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=dict(case), seed=(int(seed) * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 64), offset=int(seed) % 1000)
    if c["op"] == "quantise":
        s["x"] = _normal(g, c["rows"], c["cols"], DTYPE[c["dtype"]])
        s["scale"] = _scale_of(s["x"]) if c["fmt"] == "nvfp4" else None
    elif c["op"] == "dropout":
        s["x"] = _normal(g, c["rows"], c["cols"], DTYPE[c["dtype"]])
        s["residual"] = _normal(g, c["rows"], c["cols"], DTYPE[c["dtype"]]) if c["residual"] else None
    elif c["op"] == "product":
        s["a"] = _held(g, c["m"], c["k"], c["fmt"])
        s["b"] = _held(g, c["n"], c["k"], c["fmt"])
    elif c["op"] == "tokens":
        s["x"] = _normal(g, c["m"], c["k"], DTYPE[c["dtype"]])
        s["w"] = _held(g, c["n"], c["k"], c["fmt"])
    else:
        dt = DTYPE[c["dtype"]]
        s["x"] = _normal(g, c["tokens"], c["inputs"], dt)
        s["w"] = (torch.randn((c["outputs"], c["inputs"]), generator=g, device="cuda")
                  / math.sqrt(c["inputs"])).to(dt)
        s["dy"] = (torch.randn((c["tokens"], c["outputs"]), generator=g, device="cuda") / 16).to(dt)
    return s


# ------------------------------------------------------------------ plain form
def _bits16(rows, cols, seed, offset, purpose):
    """The 16 random bits of every element, as int64."""
    groups = (cols + 7) // 8
    mask = 0xFFFFFFFF
    c0 = torch.arange(groups, device="cuda").view(1, -1).expand(rows, groups)
    c1 = torch.arange(rows, device="cuda").view(-1, 1).expand(rows, groups)
    c2 = torch.full_like(c0, offset & mask)
    c3 = torch.full_like(c0, ((offset >> 32) & 0x7FFFFFFF) | (purpose << 31))
    k0, k1 = seed & mask, (seed >> 32) & mask
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & mask) ^ c1 ^ k0, p1 & mask, ((p0 >> 32) & mask) ^ c3 ^ k1, p0 & mask)
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    w = torch.stack([c0, c1, c2, c3], dim=-1)
    return torch.stack([w & 0xFFFF, w >> 16], dim=-1).reshape(rows, groups * 8)[:, :cols]


def _drop(x, p, seed, offset):
    """FP32 dropout: kept values times 65536 / (how many of 65536 are kept)."""
    kept = math.floor((1 - p) * 65536 + 0.5)
    if kept == 65536:
        return x
    keep = _bits16(x.shape[0], x.shape[1], seed, offset, 0) < kept
    return torch.where(keep, x * np.float32(65536 / max(kept, 1)), 0.0)


def _quantise(x, fmt, rounding, bits, gs):
    """4-bit codes (a byte each, rows padded to whole blocks) and scale bytes of FP32 x."""
    block = BLOCK[fmt]
    rows, cols = x.shape
    pad = -cols % block
    x = torch.nn.functional.pad(x, (0, pad))
    xb = x.view(rows, -1, block)
    a = xb.abs().amax(-1)
    whole = torch.isfinite(xb).all(-1)
    if fmt == "mxfp4":
        word = a.view(torch.int32)
        e = (word >> 23) - 2
        if rounding == "stochastic":
            e = e + ((word & 0x7FFFFF) > 0x400000).int()
        e = e.clamp(0, 254)
        inverse = ((254 - e) << 23).view(torch.float32)
        scales = torch.where(whole, e, 255).to(torch.uint8)
    else:
        six = gs * torch.full_like(gs, 6.0)
        s8 = (a / six).clamp(max=448.0).to(torch.float8_e4m3fn)
        if rounding == "stochastic":
            up = (six * s8.float() < a) & (s8.view(torch.uint8) < 0x7E)
            s8 = (s8.view(torch.uint8) + up.to(torch.uint8)).view(torch.float8_e4m3fn)
        d = (s8.float() * gs).unsqueeze(-1)
        scales = torch.where(whole, s8.view(torch.uint8), 0x7F).to(torch.uint8)
    v = xb * inverse.unsqueeze(-1) if fmt == "mxfp4" else torch.where(d > 0, xb / d, 0.0)
    v = v.abs().clamp(max=6.0)
    if rounding == "nearest":
        code = ((v > 0.25).byte() + (v >= 0.75).byte() + (v > 1.25).byte() + (v >= 1.75).byte()
                + (v > 2.5).byte() + (v >= 3.5).byte() + (v > 5.0).byte())
    else:  # the grid steps are 0.5 below 2, 1 below 4, 2 below 6; up with the probability of the remainder
        per = torch.where(v < 2, 2.0, torch.where(v < 4, 1.0, 0.5))
        first = torch.where(v < 2, 0, torch.where(v < 4, 2, 4))
        t = v * per
        low = t.floor()
        r = torch.nn.functional.pad(bits, (0, pad)).view(rows, -1, block)
        code = (first + low.int() + ((t - low) * 65536 >= (65536 - r).float()).int()).byte()
    code = code | ((xb < 0) & (code > 0)).byte() * 8
    return torch.where(whole.unsqueeze(-1), code, 0).to(torch.uint8).view(rows, -1), scales


def _pack(codes):
    codes = torch.nn.functional.pad(codes, (0, -codes.shape[1] % 32))
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _tile(scales):
    s = torch.nn.functional.pad(scales, (0, -scales.shape[1] % 4, 0, -scales.shape[0] % 128))
    return s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untile(tiles, rows, blocks):
    kt = (blocks + 3) // 4
    return tiles.view(-1, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kt * 4)[:rows, :blocks]


def _values(codes, scales, cols, fmt, gs):
    """FP32 values of one code per byte and of row-major scale bytes."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    if fmt == "mxfp4":
        e = scales.int()
        size = torch.where(e == 0, 2.0 ** -127, (e << 23).view(torch.float32))
        size = torch.where(e == 255, math.nan, size)
    else:
        size = scales.view(torch.float8_e4m3fn).float()
    blocks = scales.shape[1]
    v = table[codes[:, :blocks * BLOCK[fmt]].int()].view(codes.shape[0], blocks, -1) * size.unsqueeze(-1)
    v = v if gs is None else v * gs
    return v.view(codes.shape[0], -1)[:, :cols]


def _expand(held, cols, fmt, with_gs=True):
    packed, tiles, gs = held
    codes = torch.stack([packed & 15, packed >> 4], dim=-1).view(packed.shape[0], -1)
    scales = _untile(tiles, packed.shape[0], math.ceil(cols / BLOCK[fmt])).contiguous()
    return _values(codes, scales, cols, fmt, gs if with_gs else None)


def _plain_quantise(s):
    c = s["case"]
    x = _drop(s["x"].float(), c["p"], s["seed"], s["offset"])
    bits = _bits16(x.shape[0], x.shape[1], s["seed"], s["offset"], 1) if c["rounding"] == "stochastic" else None
    out = {}
    if c["transposed"] != "only":
        q = _quantise(x, c["fmt"], c["rounding"], bits, s["scale"])
        out["rows"] = _values(*q, x.shape[1], c["fmt"], s["scale"]).to(torch.bfloat16)
    if c["transposed"] != "no":
        bits = bits.t().contiguous() if bits is not None else None
        q = _quantise(x.t().contiguous(), c["fmt"], c["rounding"], bits, s["scale"])
        out["columns"] = _values(*q, x.shape[0], c["fmt"], s["scale"]).to(torch.bfloat16)
    return out


def _plain_step(s):
    c, dt = s["case"], DTYPE[s["case"]["dtype"]]
    seed, offset, fmt = s["seed"], s["offset"], "mxfp4"

    def both(x, rounding, bits):
        t, u = x.t().contiguous(), bits.t().contiguous() if bits is not None else None
        return (_values(*_quantise(x, fmt, rounding, bits, None), x.shape[1], fmt, None),
                _values(*_quantise(t, fmt, rounding, u, None), x.shape[0], fmt, None))

    x, xt = both(_drop(s["x"].float(), c["p"], seed, offset), "nearest", None)
    w, wt = both(s["w"].float(), "nearest", None)
    dy, dyt = both(s["dy"].float(), "stochastic", _bits16(c["tokens"], c["outputs"], seed, offset, 1))
    return dict(y=(x @ w.t()).to(dt), dx=_drop(dy @ wt.t(), c["p"], seed, offset).to(dt), dw=dyt @ xt.t())


def _plain(s):
    c = s["case"]
    if c["op"] == "quantise":
        return _plain_quantise(s)
    if c["op"] == "dropout":
        y = _drop(s["x"].float(), c["p"], s["seed"], s["offset"])
        y = y if s["residual"] is None else y + s["residual"].float()
        return y.to(s["x"].dtype)
    if c["op"] == "product":
        return (_expand(s["a"], c["k"], c["fmt"]) @ _expand(s["b"], c["k"], c["fmt"]).t()).to(DTYPE[c["out"]])
    if c["op"] == "tokens":
        return (s["x"].float() @ _expand(s["w"], c["k"], c["fmt"]).t()).to(s["x"].dtype)
    return _plain_step(s)


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import precision_tensor_core_gb300 as ptc

    c = s["case"]
    if c["op"] == "quantise":
        q = ptc.quantize_fp4(s["x"], c["fmt"], transposed={"no": False, "only": True, "both": "both"}[c["transposed"]],
                             rounding=c["rounding"], tensor_scale=s["scale"], p=c["p"], seed=s["seed"],
                             offset=s["offset"])
        if c["transposed"] == "both":
            return {"rows": ptc.dequantize_fp4(q[0]), "columns": ptc.dequantize_fp4(q[1])}
        return {"rows" if c["transposed"] == "no" else "columns": ptc.dequantize_fp4(q)}
    if c["op"] == "dropout":
        return ptc.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])
    if c["op"] == "product":
        a, b = (ptc.Fp4Matrix(*s[m][:2], c["k"], c["fmt"], s[m][2]) for m in "ab")
        return ptc.matmul_fp4(a, b, out_dtype=DTYPE[c["out"]])
    if c["op"] == "tokens":
        w = ptc.Fp4Matrix(*s["w"][:2], c["k"], c["fmt"], s["w"][2])
        return ptc.matmul_a16_fp4(s["x"], w)
    from precision_tensor_core_gb300 import fp4_linear

    y, saved = fp4_linear.forward(s["x"], s["w"], p=c["p"], seed=s["seed"], offset=s["offset"])
    dx, dw = fp4_linear.backward(s["dy"], saved)
    return dict(y=y, dx=dx, dw=dw)


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_bits(rows, cols, seed, offset, purpose):
    """Philox4x32-10 on the host; 16 bits per element, as float64 on the GPU."""
    m32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    groups = -(-cols // 8)
    col, row = np.meshgrid(np.arange(groups, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    ctr = [col, row, np.full_like(col, offset % 2**32), np.full_like(col, offset // 2**32 % 2**31 + purpose * 2**31)]
    key = [seed % 2**32, seed // 2**32]
    for _ in range(10):
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> sh) ^ ctr[1] ^ np.uint64(key[0]), b & m32, (a >> sh) ^ ctr[3] ^ np.uint64(key[1]), a & m32]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    out = np.empty((rows, groups, 8), dtype=np.int32)
    for j in range(4):
        out[:, :, 2 * j] = ctr[j] % np.uint64(65536)
        out[:, :, 2 * j + 1] = ctr[j] // np.uint64(65536)
    return torch.from_numpy(out.reshape(rows, groups * 8)[:, :cols].copy()).cuda().double()


def _exact_drop(x, p, seed, offset):
    kept = int((1 - p) * 65536 + 0.5)
    if kept >= 65536:
        return x
    y = x * (65536.0 / max(1, kept))
    return y.masked_fill(_exact_bits(*x.shape, seed, offset, 0) >= kept, 0.0)


def _exact_e4m3(v):
    """Nearest E4M3 number, ties to even, at most 448."""
    _, e = torch.frexp(v)
    step = torch.pow(2.0, (e - 1).clamp(min=-6).double() - 3)
    return ((v / step).round() * step).clamp(max=448.0)


def _exact_quantised(x, fmt, rounding, u, gs):
    """The values a quantised matrix stands for, in 64 bits (finite inputs)."""
    rows, cols = x.shape
    n = 32 if fmt == "mxfp4" else 16
    blocks = -(-cols // n)
    full = x.new_zeros((rows, blocks * n))
    full[:, :cols] = x
    full = full.reshape(rows, blocks, n)
    big = full.abs().max(-1, keepdim=True).values
    if fmt == "mxfp4":
        m, e = torch.frexp(big)  # big = m * 2^e, 0.5 <= m < 1
        e = e.double() - 3
        if rounding == "stochastic":
            e = torch.where(m > 0.75, e + 1, e)
        d = torch.pow(2.0, torch.where(big > 0, e, -127.0).clamp(min=-127.0))
    else:
        g = gs.double().item()
        s = _exact_e4m3(big / (6 * g))
        if rounding == "stochastic":
            _, e = torch.frexp(s)
            step = torch.pow(2.0, (e - 1).clamp(min=-6).double() - 3)
            s = torch.where((s * 6 * g < big) & (s < 448), s + step, s)
        d = s * g
    v = torch.where(d > 0, full.abs() / d, 0.0).clamp(max=6.0)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    at = torch.searchsorted(grid, v, right=True) - 1  # the last grid value not above v
    low, high = grid[at], grid[(at + 1).clamp(max=7)]
    if rounding == "nearest":
        middle = (low + high) / 2
        up = (v > middle) | ((v == middle) & (at % 2 == 1) & (at < 7))
    else:
        r = x.new_zeros((rows, blocks * n))
        r[:, :cols] = u
        gap = torch.where(high > low, high - low, 1.0)
        up = (v - low) / gap + r.reshape(rows, blocks, n) / 65536 >= 1
    out = torch.where(up, high, low) * d * torch.sign(full)
    return out.reshape(rows, -1)[:, :cols]


def _exact_held(held, cols, fmt):
    """Values of packed codes and tiled scales, element by element from the layout."""
    packed, tiles, gs = held
    rows, n = packed.shape[0], 32 if fmt == "mxfp4" else 16
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    k = torch.arange(cols, device="cuda")
    nibble = (packed[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
    v = grid[nibble & 7] * (1 - 2 * (nibble >> 3)).double()
    r, b = torch.arange(rows, device="cuda").view(-1, 1), torch.arange(-(-cols // n), device="cuda").view(1, -1)
    per_row = (-(-cols // n) + 3) // 4
    byte = tiles[((r // 128) * per_row + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4].double()
    if fmt == "mxfp4":
        size = torch.pow(2.0, byte - 127)
    else:
        e, m = torch.div(byte, 8, rounding_mode="floor") % 16, byte % 8
        size = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, e - 7)) * gs.double()
    return v * size[:, k // n]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "product":
        return _exact_held(s["a"], c["k"], c["fmt"]) @ _exact_held(s["b"], c["k"], c["fmt"]).t()
    if c["op"] == "tokens":
        return s["x"].double() @ _exact_held(s["w"], c["k"], c["fmt"]).t()
    if c["op"] == "dropout":
        y = _exact_drop(s["x"].double(), c["p"], s["seed"], s["offset"])
        return y if s["residual"] is None else y + s["residual"].double()
    if c["op"] == "quantise":
        x = _exact_drop(s["x"].double(), c["p"], s["seed"], s["offset"])
        u = _exact_bits(*x.shape, s["seed"], s["offset"], 1) if c["rounding"] == "stochastic" else None
        out = {}
        if c["transposed"] != "only":
            out["rows"] = _exact_quantised(x, c["fmt"], c["rounding"], u, s["scale"])
        if c["transposed"] != "no":
            out["columns"] = _exact_quantised(x.t(), c["fmt"], c["rounding"], None if u is None else u.t(), s["scale"])
        return out
    x = _exact_drop(s["x"].double(), c["p"], s["seed"], s["offset"])
    w, dy = s["w"].double(), s["dy"].double()
    u = _exact_bits(*dy.shape, s["seed"], s["offset"], 1)
    near, some = ("mxfp4", "nearest", None, None), ("mxfp4", "stochastic")
    y = _exact_quantised(x, *near) @ _exact_quantised(w, *near).t()
    dx = _exact_quantised(dy, *some, u, None) @ _exact_quantised(w.t(), *near).t()
    dw = _exact_quantised(dy.t(), *some, u.t(), None) @ _exact_quantised(x.t(), *near).t()
    return dict(y=y, dx=_exact_drop(dx, c["p"], s["seed"], s["offset"]), dw=dw)
