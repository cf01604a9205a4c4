"""A linear layer whose products run in microscaled 4 bits: y = dropout(x) W^T.

    python -m precision_tensor_core_gb300.fp4_linear --tokens 4096 --inputs 2048 --outputs 8192

The training step quantises x (after dropout, without storing the mask), W and
the gradient once each, along both axes in one pass, since the three products
contract over different axes:

    y  = q(dropout(x)) . q(W)^T          contraction over inputs
    dx = dropout'(q(dy) . q(W))          over outputs: the columns of W
    dW = q(dy)^T . q(dropout(x))         over tokens: the columns of dy and x

x and W are rounded to nearest, dy stochastically, so that the rounding of the
gradients has no bias (beyond 2^-16 of the gap between codes).  decode() is the serving form of a few tokens: 16-bit
activations with the 4-bit weights, read once.  The master weights stay with
the caller.  Both passes are explicit and outside autograd: forward() and
backward() take tensors that require grad as they are, and their results do not.
"""
from __future__ import annotations

import argparse

from . import dropout, matmul_a16_fp4, matmul_fp4, quantize_fp4

FORMAT = "mxfp4"


def forward(x, w, p=0.0, seed=0, offset=0):
    """y (tokens, outputs) of x (tokens, inputs) and w (outputs, inputs), and what
    backward() needs."""
    import torch
    with torch.no_grad():
        xq, xqt = quantize_fp4(x, FORMAT, transposed="both", p=p, seed=seed, offset=offset)
        wq, wqt = quantize_fp4(w, FORMAT, transposed="both")
        y = matmul_fp4(xq, wq, out_dtype=x.dtype)
    return y, (xqt, wqt, p, seed, offset)


def backward(dy, saved):
    """(dx in dy's dtype, dW in float32) of the gradient dy (tokens, outputs).  The
    rounding bits of dy come from the step's seed and offset, in a stream of
    their own."""
    import torch
    xqt, wqt, p, seed, offset = saved
    with torch.no_grad():
        dyq, dyqt = quantize_fp4(dy, FORMAT, transposed="both", rounding="stochastic", seed=seed, offset=offset)
    if p > 0.0:  # (the product stays in FP32, so that dx is rounded once)
        dx = dropout(matmul_fp4(dyq, wqt, out_dtype=torch.float32), p, seed, offset, out_dtype=dy.dtype)
    else:
        dx = matmul_fp4(dyq, wqt, out_dtype=dy.dtype)
    return dx, matmul_fp4(dyqt, xqt, out_dtype=torch.float32)


def decode(x, wq):
    """y of a few tokens x (up to 16 rows of 16-bit activations) and quantised weights."""
    return matmul_a16_fp4(x, wq)


def main():
    import torch

    from . import PTC_OK, gemm_poll_device_error

    a = argparse.ArgumentParser(description="One training step and one decoding step on random data.")
    for name, value in (("tokens", 4096), ("inputs", 2048), ("outputs", 8192)):
        a.add_argument("--" + name, type=int, default=value)
    a.add_argument("--p", type=float, default=0.1)
    a = a.parse_args()
    torch.manual_seed(0)
    x = torch.randn(a.tokens, a.inputs, device="cuda").bfloat16()
    w = (torch.randn(a.outputs, a.inputs, device="cuda") / a.inputs ** 0.5).bfloat16()
    dy = torch.randn(a.tokens, a.outputs, device="cuda").bfloat16()
    y, saved = forward(x, w, p=a.p, seed=1, offset=0)
    dx, dw = backward(dy, saved)
    xd = dropout(x, a.p, 1, 0).float()
    for name, got, want in (("y", y, xd @ w.float().t()),
                            ("dx", dx, dropout((dy.float() @ w.float()).bfloat16(), a.p, 1, 0).float()),
                            ("dW", dw, dy.float().t() @ xd)):
        print(f"{name}: {tuple(got.shape)} {got.dtype}, off the unquantised product by "
              f"{((got.float() - want).norm() / want.norm()).item():.3f} of its norm")
    few = decode(x[:4], quantize_fp4(w, FORMAT))
    print(f"decode: {tuple(few.shape)} {few.dtype}, off by "
          f"{((few.float() - x[:4].float() @ w.float().t()).norm() / few.float().norm()).item():.3f}")
    assert gemm_poll_device_error() == PTC_OK


if __name__ == "__main__":
    main()
