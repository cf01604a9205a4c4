"""The gradient's ring of rows with several rows per CTA: in place, and with threads past the rows' end."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.test_gpu_norm import F32, TYPES, least, rand, ulp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def reference(dy, s, w, ds, eps=1e-6):
    """dx, the size of its terms, dweight and the size of its terms, in 64 bits."""
    v, d = s.double(), dy.double()
    r = (v.square().mean(1, keepdim=True) + eps).rsqrt()
    g, u = d * w.double(), v * r
    dx = r * (g - u * (g * u).mean(1, keepdim=True)) + ds.double()
    return dx, r * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True)) + ds.double().abs(), (d * u).sum(0), (d * u).abs().sum(0)


def check(got, want, dtype, rows):
    dx, size, dw, size_w = want
    bound = ulp(dtype) * (dx.abs() + F32 * size) + F32 * size + least(dtype)
    assert bool(((got[0].double() - dx).abs() <= bound).all())
    # (at most rows / 8 of a CTA's or share's terms in a row, and 40 additions more)
    assert bool(((got[1].double() - dw).abs() <= (F32 + (rows / 8 + 40) * 2.0 ** -24) * size_w + 1e-30).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, cols", [(700, 1), (700, 3), (700, 7), (5000, 9), (700, 101), (3000, 250), (700, 1023), (700, 2049), (1300, 5003),
                                        (700, 8191), (650, 9001)])
def test_threads_past_the_rows_end(rows, cols, dtype):
    """Rows of odd length one after the other begin at every element of a word; the threads of a CTA are a multiple of
    32, those past a row's end bring zeros."""
    dy, s, ds, w = (rand(k, *shape, dtype=dtype) for k, shape in enumerate([(rows, cols)] * 3 + [(cols,)]))
    got = ptc.rms_norm_backward(dy, s, w, dsum=ds)
    check(got, reference(dy, s, w, ds), dtype, rows)
    again = ptc.rms_norm_backward(dy, s, w, dsum=ds)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("rows, cols", [(700, 96), (700, 101), (3000, 96), (3000, 101), (2000, 5003), (1300, 9000), (1300, 9001), (700, 20001)])
def test_in_place_with_many_rows(rows, cols, which, dtype):
    """dx over dy, s or dsum while other rows are on their way to the same CTA, and while other CTAs read the words
    that a row shares with its neighbour: bit for bit what separate memory gives."""
    t = [rand(i, rows, cols, dtype=dtype) for i in range(3)]
    w = rand(5, cols, dtype=dtype)
    want = ptc.rms_norm_backward(t[0], t[1], w, dsum=t[2])
    check(want, reference(t[0], t[1], w, t[2]), dtype, rows)
    for _ in range(3):
        held = [x.clone() for x in t]
        got = ptc.rms_norm_backward(held[0], held[1], w, dsum=held[2], out=held[which])
        assert got[0] is held[which] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
