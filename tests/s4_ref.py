"""A plain reference of grouped 4-bit integer weights, in 64 bits, and inputs for it."""
import torch

from tests.gpu_util import DEV


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def rand(seed, *shape, dtype=torch.float32, size=1.0):
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * size).to(dtype)


def weights(seed, lead, rows, K, group, zeros=False, dtype=torch.bfloat16, slack=0):
    """Random codes of every value with scales of both signs: dict(codes, scales, zeros) row-major, values in 64 bits.
    The bytes past a row's codes, and a last odd nibble, hold anything.  slack: bytes between rows beyond the least."""
    g = gen(seed)
    lead = tuple(lead)
    groups, width = -(-K // group), -(-K // 32) * 16 + 16 * slack
    codes = torch.randint(0, 256, (*lead, rows, width), generator=g, device=DEV, dtype=torch.uint8)
    scales = (torch.randn(*lead, rows, groups, generator=g, device=DEV) * 0.1).to(dtype)
    z = (torch.randn(*lead, rows, groups, generator=g, device=DEV) * 3).to(dtype) if zeros else None
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*lead, rows, -1)[..., :K].long()
    c = torch.where(nib > 7, nib - 16, nib).double()
    at = torch.arange(K, device=DEV) // group
    raw = c if z is None else c - z.double()[..., at]
    return dict(codes=codes, scales=scales, zeros=z, group=group, K=K, values=raw * scales.double()[..., at],
                # what an element's products are taken of: codes + 8 up to 15, and 8 + z
                size=(c + 8 + (8.0 if z is None else (8 + z.double()[..., at]).abs())) * scales.double()[..., at].abs())


def matrix(w):
    import precision_tensor_core_gb300 as ptc
    return ptc.S4Matrix(w["codes"], ptc.S4Matrix.tile_scales(w["scales"]), w["K"], w["group"],
                        None if w["zeros"] is None else ptc.S4Matrix.tile_scales(w["zeros"]))


def check(got, x, w, dtype, extra=0.0):
    """Products are exact; a tensor-core sum of a block takes at most 32 steps that each lose up to 2^-22 of what they
    hold (the sums' alignment is truncated), joining blocks and shares rounds a few more times: below 2^-17 of the
    products' magnitudes; then the type's rounding."""
    want = x.double() @ w["values"].t()
    size = x.double().abs() @ w["size"].t()
    bound = torch.finfo(dtype).eps / 2 * want.abs() + (2.0 ** -17) * size + extra + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert got.dtype == dtype and got.shape == want.shape
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), (off / bound).max()
