"""Performance cases of the operators around quantised products: root-mean-square
norm (with the residual's addition, in the input's type or in 8 bits with a scale
per row, and its gradient), the product of a few 16-bit tokens with 4-bit integer
weights that have group scales, and a whole mixture-of-experts layer with such
weights for a few tokens.

Each case is computed either in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, by the calls a
user makes of the library.  ``exact`` gives the same outputs from the
operators' definitions in 64 bits.

Definitions.
  norm      s = x + residual, rounded to x's type (the residual stream that is
            stored); r = 1 / sqrt(mean(s^2) + eps) per row; y = s r weight.
            In 8 bits: t = s weight, a = max |t| of the row, codes 127 t / a
            rounded to nearest (ties to even), row scale a r / 127.
  gradient  g = dy weight; dx = r (g - s r^2 mean(g s)) + dsum, dweight the sum over
            rows of dy s r.
  weights   code c in -8 .. 7 (two's complement, two per byte, the even element
            in the low nibble), scale s and zero z (0 where there are none) per row
            and group of `group` elements: (c - z) s.  Scales and zeros are 16-bit
            numbers in tiles: [row / 16][group][row % 16].
  experts   logits = x router^T; the top_k largest of a token (ties to the lowest
            index), their weights p the softmax over all logits, divided by their
            sum where `renormalize`; y = sum of p down (silu(gate x) * (up x)).
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decoding one sequence: the residual's addition and the norm before a block; latency counts
        dict(name="norm of one token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, bits=16),
        # the same of a training batch or a long prompt
        dict(name="norm of a batch", op="norm", rows=8192, cols=8192, dtype="bf16", residual=True, bits=16),
        # activations of a ragged prompt for an 8-bit product, odd sizes
        dict(name="norm to 8 bits", op="norm", rows=2047, cols=5003, dtype="f16", residual=False, bits=8),
        # the backward pass of a batch, with the residual stream's own gradient
        dict(name="norm gradient", op="gradient", rows=8192, cols=8192, dtype="bf16", dsum=True),
        # the backward pass of a small FP32 layer with odd sizes
        dict(name="norm gradient small", op="gradient", rows=333, cols=777, dtype="f32", dsum=False),
        # decoding one sequence: a square layer, read once
        dict(name="one token", op="product", m=1, n=4096, k=4096, group=128, zeros=False, dtype="bf16"),
        # decoding a batch of sequences against a wide layer whose codes have zero points
        dict(name="sixteen tokens", op="product", m=16, n=16384, k=8192, group=128, zeros=True, dtype="f16"),
        # a few drafted tokens against a layer of uneven sizes, small groups, the last one partial
        dict(name="ragged product", op="product", m=5, n=1339, k=2090, group=32, zeros=True, dtype="bf16"),
        # decoding one sequence through a layer of many small experts
        dict(name="experts, one token", op="experts", tokens=1, hidden=2048, inner=1024, experts=64, top_k=8,
             group=128, zeros=False, renormalize=True, dtype="bf16"),
        # decoding a batch of sequences through a layer of large experts, most of them active
        dict(name="experts, sixteen tokens", op="experts", tokens=16, hidden=4096, inner=2048, experts=32, top_k=4,
             group=128, zeros=False, renormalize=False, dtype="bf16"),
        # odd sizes throughout, small groups with zero points
        dict(name="experts, ragged", op="experts", tokens=7, hidden=1000, inner=333, experts=13, top_k=3,
             group=32, zeros=True, renormalize=True, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "gradient", "gradient", "product", "product", "product", "experts",
                     "experts", "experts"])
    if op in ("norm", "gradient"):
        rows = _log(rng, 1, 8192)
        cols = _log(rng, 16, 16384 if rows <= 4096 else 8192)
        dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        if dtype == "f32":  # (as many bytes as the largest listed case has)
            rows = min(rows, 2048)
        if op == "norm":
            bits = rng.choice([16, 16, 8])
            if bits == 8:  # (16-bit activations)
                rows, cols, dtype = min(rows, 2047), min(cols, 5003), rng.choice(["bf16", "f16"])
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.choice([True, False]), bits=bits)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, dsum=rng.choice([True, False]))
    group, zeros = rng.choice([32, 64, 128, 128, 256]), rng.choice([True, False])
    dtype = rng.choice(["bf16", "f16"])
    if op == "product":
        return dict(op=op, m=rng.choice([1, rng.randint(1, 4), rng.randint(1, 16)]), n=_log(rng, 64, 16384),
                    k=_log(rng, 64, 8192), group=group, zeros=zeros, dtype=dtype)
    c = dict(op=op, tokens=_log(rng, 1, 32), hidden=_log(rng, 128, 4096), inner=_log(rng, 64, 2048),
             experts=_log(rng, 4, 128), top_k=rng.randint(1, 8), group=group, zeros=zeros,
             renormalize=rng.choice([True, False]), dtype=dtype)
    while c["tokens"] * c["experts"] * c["hidden"] * c["inner"] > 16 * 32 * 4096 * 2048 or \
            c["experts"] * c["hidden"] * c["inner"] > 32 * 4096 * 2048:
        c["experts"] = max(4, c["experts"] // 2)
        c["tokens"] = max(1, c["tokens"] - 3)
    c["top_k"] = min(c["top_k"], c["experts"])
    return c


def work(case):
    c, size = case, {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]

    def held(rows, cols):  # codes, scales, zeros
        return rows * cols / 2 + rows * math.ceil(cols / c["group"]) * (4 if c["zeros"] else 2)

    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        out = size if c["bits"] == 16 else 1 + 4  # (codes, and the values they stand for)
        return dict(bytes=n * (size * (3 if c["residual"] else 1) + out) + c["cols"] * size, flops=5 * n)
    if c["op"] == "gradient":
        n = c["rows"] * c["cols"]
        return dict(bytes=n * size * (4 if c["dsum"] else 3) + c["cols"] * (size + 4), flops=10 * n)
    if c["op"] == "product":
        return dict(bytes=held(c["n"], c["k"]) + 2 * c["m"] * (c["n"] + c["k"]), flops=2 * c["m"] * c["n"] * c["k"])
    t, d, i, e, k = c["tokens"], c["hidden"], c["inner"], c["experts"], c["top_k"]
    active = e * (1 - (1 - k / e) ** t)  # experts that some token chooses, on average
    return dict(bytes=active * (held(2 * i, d) + held(d, i)) + 2 * e * d + 4 * t * d,
                flops=6 * t * k * i * d + 2 * t * e * d)


# ------------------------------------------------------------------ inputs
def _normal(g, rows, cols, dtype):
    """Activations: normal values with a spread of channel sizes and a few large channels."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    size = torch.exp(0.5 * torch.randn((1, cols), generator=g, device="cuda"))
    size = torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.01, size * 10, size)
    return (x * size).to(dtype)


def _tile(rows):
    """(..., rows, groups) to [..., row / 16, group, row % 16], flat."""
    r, n = rows.shape[-2:]
    t = torch.nn.functional.pad(rows, (0, 0, 0, -r % 16))
    return t.reshape(*rows.shape[:-2], -1, 16, n).transpose(-1, -2).contiguous().view(-1)


def _weights(g, shape, cols, group, zeros, dtype):
    """Normal weights rounded to 4-bit codes, as a program has them in hand: codes
    (rows of a multiple of 16 bytes), tiled scales and zeros."""
    groups = -(-cols // group)
    w = torch.randn((*shape, cols), generator=g, device="cuda") / math.sqrt(cols)
    w = torch.nn.functional.pad(w, (0, groups * group - cols)).view(*shape, groups, group)
    if zeros:
        low, high = w.amin(-1), w.amax(-1)
        scale = ((high - low) / 15).to(dtype)
        zero = (-8 - low / scale.float()).round().clamp(-8, 7).to(dtype)
    else:
        scale, zero = (w.abs().amax(-1) / 7).to(dtype), None
    code = w / scale.float().unsqueeze(-1)
    code = code if zero is None else code + zero.float().unsqueeze(-1)
    code = code.round().clamp(-8, 7).to(torch.int8).view(*shape, -1)[..., :cols].view(torch.uint8) & 15
    code = torch.nn.functional.pad(code, (0, -cols % 32))
    return dict(codes=code[..., 0::2] | (code[..., 1::2] << 4), scales=_tile(scale),
                zeros=None if zero is None else _tile(zero))


def prepare(case, seed):
    c, dt = case, DTYPE[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=dict(case))
    if c["op"] in ("norm", "gradient"):
        s["x"] = _normal(g, c["rows"], c["cols"], dt)
        s["weight"] = (1 + 0.2 * torch.randn(c["cols"], generator=g, device="cuda")).to(dt)
        if c.get("residual"):
            s["residual"] = _normal(g, c["rows"], c["cols"], dt)
        if c["op"] == "gradient":
            s["dy"] = (torch.randn((c["rows"], c["cols"]), generator=g, device="cuda") / 16).to(dt)
            s["dsum"] = (torch.randn((c["rows"], c["cols"]), generator=g, device="cuda") / 16).to(dt) if c["dsum"] else None
    elif c["op"] == "product":
        s["x"] = _normal(g, c["m"], c["k"], dt)
        s["w"] = _weights(g, (c["n"],), c["k"], c["group"], c["zeros"], dt)
    else:
        s["x"] = _normal(g, c["tokens"], c["hidden"], dt)
        s["router"] = (torch.randn((c["experts"], c["hidden"]), generator=g, device="cuda")
                       / math.sqrt(c["hidden"])).to(dt)
        s["gate_up"] = _weights(g, (c["experts"], 2 * c["inner"]), c["hidden"], c["group"], c["zeros"], dt)
        s["down"] = _weights(g, (c["experts"], c["hidden"]), c["inner"], c["group"], c["zeros"], dt)
    return s


# ------------------------------------------------------------------ plain form
def _values(w, rows, cols, group):
    """FP32 values of packed codes with tiled scales."""
    lead = w["codes"].shape[:-2]
    groups = -(-cols // group)

    def per_element(t):
        t = t.view(*lead, -1, groups, 16).transpose(-1, -2).reshape(*lead, -1, groups)[..., :rows, :]
        return t.float().repeat_interleave(group, dim=-1)[..., :cols]

    c = torch.stack([w["codes"] & 15, w["codes"] >> 4], dim=-1).view(*lead, rows, -1)[..., :cols].float()
    c = torch.where(c > 7, c - 16, c)
    c = c if w["zeros"] is None else c - per_element(w["zeros"])
    return c * per_element(w["scales"])


def _plain_norm(s):
    c, x = s["case"], s["x"]
    total = x if not c["residual"] else (x.float() + s["residual"].float()).to(x.dtype)
    v, w = total.float(), s["weight"].float()
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    if c["bits"] == 16:
        out = dict(y=(v * r * w).to(x.dtype))
    else:
        t = v * w
        a = t.abs().amax(-1, keepdim=True)
        code = torch.round(t.double() * 127 / a.double()).float()  # (in 64 bits: quotients next to a border)
        out = dict(values=code * (a * r / 127))
    if c["residual"]:
        out["sum"] = total
    return out


def _plain_gradient(s):
    v, w, dy = s["x"].float(), s["weight"].float(), s["dy"].float()
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    g = dy * w
    dx = r * (g - v * r * r * (g * v).mean(-1, keepdim=True))
    dx = dx if s["dsum"] is None else dx + s["dsum"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * v * r).sum(0))


def _plain_experts(s):
    c, x = s["case"], s["x"].float()
    logits = x @ s["router"].float().t()
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = ids[:, :c["top_k"]]
    e = torch.exp(best - best[:, :1])
    p = e[:, :c["top_k"]] / (e[:, :c["top_k"]] if c["renormalize"] else e).sum(-1, keepdim=True)
    gu = x @ _values(s["gate_up"], 2 * c["inner"], c["hidden"], c["group"]).transpose(-1, -2)  # (experts, tokens, 2 inner)
    gate, up = gu[..., :c["inner"]], gu[..., c["inner"]:]
    h = gate / (1 + torch.exp(-gate)) * up
    h = h * torch.zeros_like(logits).scatter(1, ids, p).t().unsqueeze(-1)
    y = (h @ _values(s["down"], c["hidden"], c["inner"], c["group"]).transpose(-1, -2)).sum(0)
    return dict(y=y.to(s["x"].dtype), experts=ids.int(), weights=p)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "gradient":
        return _plain_gradient(s)
    if c["op"] == "product":
        return (s["x"].float() @ _values(s["w"], c["n"], c["k"], c["group"]).t()).to(s["x"].dtype)
    return _plain_experts(s)


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import precision_tensor_core_gb300 as ptc

    c = s["case"]
    if c["op"] == "norm":
        if c["bits"] == 16:
            if not c["residual"]:
                return dict(y=ptc.rms_norm(s["x"], s["weight"], EPS))
            y, total = ptc.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
            return dict(y=y, sum=total)
        got = ptc.rms_norm_s8(s["x"], s["weight"], EPS, residual=s.get("residual"))
        out = dict(values=torch.mul(got[0], got[1].unsqueeze(1)))
        if c["residual"]:
            out["sum"] = got[2]
        return out
    if c["op"] == "gradient":
        dx, dweight = ptc.rms_norm_backward(s["dy"], s["x"], s["weight"], EPS, dsum=s["dsum"])
        return dict(dx=dx, dweight=dweight)

    def matrix(w, k):
        return ptc.S4Matrix(w["codes"], w["scales"], k, c["group"], w["zeros"])

    if c["op"] == "product":
        return ptc.matmul_a16_s4(s["x"], matrix(s["w"], c["k"]))
    y, experts, weights = ptc.moe_a16_s4(s["x"], s["router"], matrix(s["gate_up"], c["hidden"]),
                                         matrix(s["down"], c["inner"]), c["top_k"], renormalize=c["renormalize"],
                                         return_routing=True)
    return dict(y=y, experts=experts, weights=weights)


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_values(w, rows, cols, group, at=()):
    """Values of one matrix, element by element from the layout; `at`: which expert."""
    codes = w["codes"][at]
    k = torch.arange(cols, device="cuda")
    r = torch.arange(rows, device="cuda").unsqueeze(1)
    nibble = (codes[:, k // 2].int() >> (4 * (k % 2)).int()) % 16
    c = ((nibble + 8) % 16 - 8).double()
    groups, tiles = -(-cols // group), -(-rows // 16)
    base = (at[0] if at else 0) * tiles * groups * 16
    where = base + (torch.div(r, 16, rounding_mode="floor") * groups + k // group) * 16 + r % 16
    if w["zeros"] is not None:
        c = c - w["zeros"][where].double()
    return c * w["scales"][where].double()


def _exact_experts(s):
    c, x = s["case"], s["x"].double()
    logits = x @ s["router"].double().t()
    p = torch.softmax(logits, -1)
    ids = torch.argsort(-logits, dim=-1, stable=True)[:, :c["top_k"]]
    weights = torch.gather(p, 1, ids)
    if c["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(c["experts"]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if token.numel() == 0:
            continue
        gu = x[token] @ _exact_values(s["gate_up"], 2 * c["inner"], c["hidden"], c["group"], (e,)).t()
        gate, up = gu[:, :c["inner"]], gu[:, c["inner"]:]
        out = (torch.sigmoid(gate) * gate * up) @ _exact_values(s["down"], c["hidden"], c["inner"], c["group"], (e,)).t()
        y.index_add_(0, token, out * weights[token, slot].unsqueeze(1))
    return dict(y=y, experts=ids.int(), weights=weights)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "experts":
        return _exact_experts(s)
    if c["op"] == "product":
        return s["x"].double() @ _exact_values(s["w"], c["n"], c["k"], c["group"]).t()
    w = s["weight"].double()
    if c["op"] == "gradient":
        v, dy = s["x"].double(), s["dy"].double()
        mean2 = torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / c["cols"]
        inv = (mean2 + EPS).rsqrt()
        unit = v * inv  # the normalised row, through which the gradient goes
        g = dy * w
        dx = inv * (g - unit * torch.sum(g * unit, 1, keepdim=True) / c["cols"])
        return dict(dx=dx if s["dsum"] is None else dx + s["dsum"].double(), dweight=torch.sum(dy * unit, 0))
    out, v = {}, s["x"].double()
    if c["residual"]:
        out["sum"] = v + s["residual"].double()
        v = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()  # (the stored sum is what is normalised)
    inv = (torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / c["cols"] + EPS).rsqrt()
    if c["bits"] == 16:
        out["y"] = v * inv * w
    else:  # (the row's r is left out of the quotient, whose ties it would disturb)
        t = v * w
        largest = torch.linalg.vector_norm(t, ord=math.inf, dim=1, keepdim=True)
        out["values"] = torch.round(127 * t / largest) * (largest * inv / 127)
    return out
