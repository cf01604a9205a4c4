"""The 4-bit operators on a stream that is not the caller's: whose memory results
take, and what may be released while they run.

A stream is kept busy by a bounded wait on the device (some tens of
milliseconds), so that work queued after it is pending when the calls under
test are made."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
CYCLES = 60_000_000


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def draw(seed, rows=600, cols=2048, dtype=torch.bfloat16):
    return torch.randn(rows, cols, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(dtype)


def parts(r):
    """The tensors of a result."""
    if isinstance(r, tuple):
        return [t for m in r for t in parts(m)]
    return [r.codes, r.scales] if isinstance(r, ptc.Fp4Matrix) else [r]


W = None


def operators():
    """name: (call(x, stream), inputs by seed)."""
    global W
    if W is None:
        W = ptc.quantize_fp4(draw(99, 520))
        torch.cuda.synchronize()
    return {
        "dropout": (lambda x, s: ptc.dropout(x, 0.3, 1, 2, residual=x, stream=s), draw),
        "quantize": (lambda x, s: ptc.quantize_fp4(x, stream=s), draw),
        "quantize both": (lambda x, s: ptc.quantize_fp4(x, "nvfp4", transposed="both", stream=s), draw),
        "dequantize": (lambda q, s: ptc.dequantize_fp4(q, stream=s), lambda seed: ptc.quantize_fp4(draw(seed))),
        "product": (lambda q, s: ptc.matmul_fp4(q, W, stream=s), lambda seed: ptc.quantize_fp4(draw(seed))),
        "few tokens": (lambda x, s: ptc.matmul_a16_fp4(x, W, stream=s), lambda seed: draw(seed, 600)),
    }


NAMES = ["dropout", "quantize", "quantize both", "dequantize", "product", "few tokens"]


@pytest.fixture(params=NAMES)
def op(request):
    call, make = operators()[request.param]
    want = [t.clone() for t in parts(call(make(1), None))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(make(1), side)  # (first use of the stream)
    torch.cuda.synchronize()
    return call, make, want, side


def same(got, want):
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(parts(got), want))


def test_results_take_no_memory_that_the_callers_stream_still_writes(op):
    call, make, want, side = op
    x = make(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    old = [torch.empty_like(t).fill_(7) for t in want]  # pending writes ...
    del old                                              # ... to memory that may be handed out again
    got = call(x, side)
    assert same(got, want)


def test_inputs_may_be_released_while_the_other_stream_runs(op):
    call, make, want, side = op
    x = make(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    got = call(x, side)
    sizes = [torch.empty_like(t) for t in parts(x)] if isinstance(x, ptc.Fp4Matrix) else [torch.empty_like(x)]
    shapes = [(t.shape, t.dtype) for t in sizes]
    del x, sizes
    garbage = [torch.empty(s, dtype=d, device=DEV).fill_(3) for s, d in shapes for _ in range(3)]
    assert same(got, want) and garbage


def test_results_may_be_released_while_the_callers_stream_reads_them(op):
    call, make, want, side = op
    x, other = make(1), make(2)
    torch.cuda.synchronize()
    got = call(x, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(CYCLES)
    copies = [t.clone() for t in parts(got)]
    del got
    later = [call(other, side) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)) and later


def test_stream_arguments():
    """Handles, the default stream by its names, and the current stream are all taken."""
    x = draw(5)
    want = ptc.dropout(x, 0.3, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (None, 0, 1, side, side.cuda_stream, torch.cuda.current_stream(), torch.cuda.default_stream()):
        y = ptc.dropout(x, 0.3, 1, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        with torch.cuda.stream(side):
            z = ptc.dropout(x, 0.3, 1, stream=s)
            assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        assert torch.equal(z, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
