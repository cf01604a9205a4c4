"""The norms and their gradient against 64-bit references.

Tolerances.  The sum of squares is FP32 in a tree of at most 64 terms in a row and 10
levels: relative error below 80 * 2^-24; 1 / rms half of that and three roundings; y two
more products: below 2^-17 in all, and the rounding to the type, eps / 2."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
F32 = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def rand(seed, *shape, dtype=torch.float32, size=1.0):
    return (torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV) * size).to(dtype)


def ulp(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def near(got, want, dtype, size=None, f32=F32):
    """got within the type's rounding of the 64-bit `want`, and f32 relative to `size`."""
    size = want.abs() if size is None else size
    bound = ulp(dtype) * (want.abs() + f32 * size) + f32 * size + least(dtype)
    off = (got.double() - want).abs() - bound
    assert got.dtype == dtype and got.shape == want.shape
    assert bool((off <= 0).all()), off.max()


def reference(s, w, eps):
    v = s.double()
    r = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    return v * r * (1.0 if w is None else w.double()), r


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 33), (2, 255), (700, 64), (700, 257), (650, 1000), (333, 1024), (7, 1025), (40, 4096),
          (1, 8192), (200, 8200), (3, 16384), (160, 16376), (3, 16385), (2, 40000), (1, 8191), (170, 5003)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_norm(rows, cols, dtype):
    x, w = rand(1, rows, cols, dtype=dtype, size=3.0), rand(2, cols, dtype=dtype)
    want, _ = reference(x, w, 1e-5)
    near(ptc.rms_norm(x, w, 1e-5), want, dtype)
    near(ptc.rms_norm(x), reference(x, None, 1e-6)[0], dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_residual(rows, cols, dtype):
    x, r, w = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype, size=20.0), rand(3, cols)
    keep = x.clone(), r.clone(), w.clone()
    y, s = ptc.rms_norm(x, w, residual=r)
    assert torch.equal(s, (x.float() + r.float()).to(dtype))
    near(y, reference(s, w, 1e-6)[0], dtype)
    assert all(torch.equal(a, b) for a, b in zip(keep, (x, r, w)))


@pytest.mark.parametrize("in_place", ["sum is residual", "sum is x", "y is x", "y is residual", "both"])
@pytest.mark.parametrize("cols", [96, 101, 20001])
def test_in_place(in_place, cols):
    x, r, w = rand(1, 50, cols, dtype=torch.bfloat16), rand(2, 50, cols, dtype=torch.bfloat16), rand(3, cols)
    want = ptc.rms_norm(x, w, residual=r)
    out = {"y is x": x, "y is residual": r, "both": x}.get(in_place)
    sum_out = {"sum is residual": r, "sum is x": x, "both": r}.get(in_place)
    y, s = ptc.rms_norm(x, w, residual=r, out=out, sum_out=sum_out)
    assert torch.equal(y, want[0]) and torch.equal(s, want[1])
    assert (out is None or y is out) and (sum_out is None or s is sum_out)


def codes_reference(s, w):
    t = s.float() if w is None else s.float() * w.float()
    a = t.abs().amax(-1, keepdim=True)
    q = torch.round(t.double() * 127 / a.double())
    return torch.where(a > 0, q, 0.0), t, a


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_s8(rows, cols, dtype, residual):
    x, w = rand(1, rows, cols, dtype=dtype, size=3.0), rand(2, cols, dtype=dtype)
    r = rand(3, rows, cols, dtype=dtype) if residual else None
    got = ptc.rms_norm_s8(x, w, 1e-5, residual=r)
    s = (x.float() + r.float()).to(dtype) if residual else x
    q, t, a = codes_reference(s, w)
    assert got[0].dtype == torch.int8 and torch.equal(got[0].double(), q)
    _, inv = reference(s, None, 1e-5)
    want = (a.double() * inv / 127).squeeze(1)
    assert bool(((got[1].double() - want).abs() <= 2.0 ** -16 * want).all())
    assert not residual or torch.equal(got[2], s)


def test_s8_borders():
    """Quotients on and next to every border, from values whose products are exact: ties go to even."""
    n = torch.arange(-254, 255, device=DEV).float()  # 127 t / a = n / 2 with a = 254
    row = torch.cat([n, torch.tensor([254.0], device=DEV)]).half()
    for k, rows in ((0, row), (1, torch.nextafter(row, torch.full_like(row, 1e4))), (2, torch.nextafter(row, -torch.full_like(row, 1e4)))):
        rows = rows.clone()
        rows[-1] = 254.0
        x = rows.repeat(3, 1)
        for c in (x, x[:, 1:]):  # aligned rows and others
            q, scale = ptc.rms_norm_s8(c)
            assert torch.equal(q.double(), codes_reference(c, None)[0]), k
    assert torch.equal(ptc.rms_norm_s8(row.unsqueeze(0))[0][0, ::2].double(), torch.round(row.double() / 2)[::2])


def test_s8_special_rows():
    x = rand(1, 9, 300, dtype=torch.bfloat16)
    x[1] = 0
    x[3, 7] = float("inf")
    x[5, 299] = float("nan")
    x[7] = 0
    x[7, 11] = -2.0 ** -130
    w = rand(2, 300, dtype=torch.float32)
    w[11] = 1.0
    q, scale = ptc.rms_norm_s8(x, w)
    ok = [0, 2, 4, 6, 8]
    assert torch.equal(q[ok], ptc.rms_norm_s8(x[ok].contiguous(), w)[0])
    assert not q[1].any() and scale[1] == 0
    assert not q[3].any() and not q[5].any() and bool(scale[[3, 5]].isnan().all())
    assert q[7, 11] == -127 and q[7].abs().sum() == 127
    y = ptc.rms_norm(x, w)
    assert torch.equal(y[ok], ptc.rms_norm(x[ok].contiguous(), w)) and not y[1].any()
    assert bool(y[5].isnan().all()) and bool(y[3, 7].isnan()) and not y[3, 8:].any()
    assert bool(ptc.rms_norm(x[1:2], eps=0.0).isnan().all())


@pytest.mark.parametrize("dtype", TYPES)
def test_views_of_one_buffer(dtype):
    """Column slices as inputs and outputs; what lies between them stays as it was."""
    buf = rand(1, 60, 1000, dtype=dtype)
    for lo, hi, at in ((0, 320, 512), (3, 330, 500), (0, 327, 512)):
        b = buf.clone()
        x, out = b[:, lo:hi], b[:, at:at + hi - lo]
        before = b.clone()
        got = ptc.rms_norm(x, out=out)  # (the order of FP32 sums goes by the rows' alignment: compared with the formula)
        near(got, reference(before[:, lo:hi], None, 1e-6)[0], dtype)
        before[:, at:at + hi - lo] = got
        assert torch.equal(b, before)
    t = buf.t()
    with pytest.raises(ValueError, match="unit column stride"):
        ptc.rms_norm(t)


def grad_reference(dy, s, w, eps, ds):
    v = s.double().requires_grad_()
    wd = (torch.ones(s.shape[1], device=DEV) if w is None else w).double().requires_grad_()
    y = v * (v.square().mean(-1, keepdim=True) + eps).rsqrt() * wd
    dx, dw = torch.autograd.grad(y, (v, wd), dy.double())
    r = (s.double().square().mean(-1, keepdim=True) + eps).rsqrt()
    g, u = dy.double() * wd.detach(), s.double() * r
    size = r * (g.abs() + u.abs() * (g.abs() * u.abs()).mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.double()
        size = size + ds.double().abs()
    return dx, dw, size, (dy.double() * u).abs().sum(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, cols", SHAPES + [(2000, 96), (1, 17000), (600, 17001)])
@pytest.mark.parametrize("dsum", [False, True])
def test_gradient(rows, cols, dtype, dsum):
    dy, s, w = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype, size=2.0), rand(3, cols, dtype=dtype)
    ds = rand(4, rows, cols, dtype=dtype) if dsum else None
    dx, dw = ptc.rms_norm_backward(dy, s, w, 1e-5, dsum=ds)
    want, want_w, size, size_w = grad_reference(dy, s, w, 1e-5, ds)
    near(dx, want, dtype, size)
    # at most 500 rows in a row (of a share), then 64 and 8 partial sums, each half an ulp
    assert dw.dtype == torch.float32 and bool(((dw.double() - want_w).abs() <= 2.0 ** -14 * size_w + 1e-30).all())
    again = ptc.rms_norm_backward(dy, s, w, 1e-5, dsum=ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("w_dtype", [None, torch.float32, torch.float16])
def test_gradient_weights(w_dtype):
    dy, s = rand(1, 37, 500, dtype=torch.float16), rand(2, 37, 500, dtype=torch.float16)
    w = None if w_dtype is None else rand(3, 500, dtype=w_dtype)
    dx, dw = ptc.rms_norm_backward(dy, s, w)
    want, want_w, size, size_w = grad_reference(dy, s, w, 1e-6, None)
    near(dx, want, torch.float16, size)
    assert bool(((dw.double() - want_w).abs() <= 2.0 ** -14 * size_w).all())


@pytest.mark.parametrize("cols", [96, 101, 20001])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_gradient_in_place(cols, which):
    t = [rand(i, 50, cols, dtype=torch.bfloat16) for i in range(3)]
    w = rand(5, cols)
    want = ptc.rms_norm_backward(t[0], t[1], w, dsum=t[2])
    got = ptc.rms_norm_backward(t[0], t[1], w, dsum=t[2], out=t[which])
    assert got[0] is t[which] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradient_of_no_rows():
    e = torch.empty(0, 40, device=DEV)
    dx, dw = ptc.rms_norm_backward(e, e, rand(1, 40))
    assert dx.shape == (0, 40) and not dw.any() and dw.shape == (40,)
    assert ptc.rms_norm(e).shape == (0, 40)
    q, scale = ptc.rms_norm_s8(torch.empty(4, 0, device=DEV))
    assert q.shape == (4, 0) and scale.shape == (4,)


def test_gradient_against_differences():
    """<dy, y(x + h v) - y(x - h v)> / 2 h of the float32 forward against <dx, v> and <dweight, v>.

    With |v| about 0.1 of |x| per element and h = 0.05 the third-order remainder is below (0.005)^2 of the value; the
    rounding 2^-22 |y| sqrt(n) / (2 h), below 1e-3 of the norms' product."""
    rows, cols = 20, 333
    x, dy, w = rand(1, rows, cols), rand(2, rows, cols), rand(3, cols)
    dx, dw = ptc.rms_norm_backward(dy, x, w)
    h = 0.05
    for seed in range(3):
        v, vw = rand(10 + seed, rows, cols, size=0.1), rand(20 + seed, cols, size=0.1)
        up, down = ptc.rms_norm(x + h * v, w), ptc.rms_norm(x - h * v, w)
        slope = (dy.double() * (up.double() - down.double())).sum() / (2 * h)
        assert abs(slope - (dx.double() * v.double()).sum()) <= 1e-3 * dx.double().norm() * v.double().norm()
        up, down = ptc.rms_norm(x, w + h * vw), ptc.rms_norm(x, w - h * vw)
        slope = (dy.double() * (up.double() - down.double())).sum() / (2 * h)
        assert abs(slope - (dw.double() * vw.double()).sum()) <= 1e-3 * dw.double().norm() * vw.double().norm()


def test_norm_to_s8_product():
    """A norm in 8 bits into the INT8 product that takes its codes and scales as they are."""
    x, r, w = rand(1, 77, 1000, dtype=torch.bfloat16), rand(2, 77, 1000, dtype=torch.bfloat16), rand(3, 1000, dtype=torch.bfloat16)
    wq = torch.randint(-127, 128, (264, 1008), generator=torch.Generator(DEV).manual_seed(4), device=DEV).to(torch.int8)[:, :1000]
    ws = rand(5, 264).abs() / 1000
    q, scale, s = ptc.rms_norm_s8(x, w, residual=r)
    y = ptc.matmul_s8_scaled(q, wq, scale, ws, out_dtype=torch.bfloat16)
    code = codes_reference(s, w)[0]
    want = (code @ wq.double().t()) * scale.double()[:, None] * ws.double()
    near(y, want, torch.bfloat16)


def test_refusals():
    x = rand(1, 6, 64, dtype=torch.bfloat16)
    bad = [
        (ValueError, lambda: ptc.rms_norm(x[0])), (ValueError, lambda: ptc.rms_norm(x, torch.ones(63, device=DEV))),
        (ValueError, lambda: ptc.rms_norm(x, torch.ones(64))), (ValueError, lambda: ptc.rms_norm(x, torch.ones(64, device=DEV).half())),
        (ValueError, lambda: ptc.rms_norm(x, eps=-1.0)), (ValueError, lambda: ptc.rms_norm(x, eps=float("nan"))),
        (ValueError, lambda: ptc.rms_norm(x, residual=x.float())), (ValueError, lambda: ptc.rms_norm(x, residual=x[:5])),
        (ValueError, lambda: ptc.rms_norm(x, out=x.float())), (ValueError, lambda: ptc.rms_norm(x, sum_out=x)),
        (ValueError, lambda: ptc.rms_norm(x, torch.ones(128, device=DEV)[::2])), (TypeError, lambda: ptc.rms_norm(x.int())),
        (ValueError, lambda: ptc.rms_norm_backward(x, x.float())), (ValueError, lambda: ptc.rms_norm_backward(x, x[:, :32])),
        (ptc.PtcError, lambda: ptc.rms_norm(x, residual=x.clone(), out=x, sum_out=x)),
        (RuntimeError, lambda: ptc.rms_norm(x.float().requires_grad_())),
        (RuntimeError, lambda: ptc.rms_norm_backward(x.float(), x.float(), torch.ones(64, device=DEV, requires_grad=True))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
    with torch.no_grad():
        ptc.rms_norm(x.float().requires_grad_())


def test_on_another_stream_and_in_a_graph():
    x, r, w = rand(1, 300, 777, dtype=torch.bfloat16), rand(2, 300, 777, dtype=torch.bfloat16), rand(3, 777)
    want = ptc.rms_norm(x, w, residual=r), ptc.rms_norm_s8(x, w), ptc.rms_norm_backward(r, x, w, dsum=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = (ptc.rms_norm(x, w, residual=r, stream=side), ptc.rms_norm_s8(x, w, stream=side),
           ptc.rms_norm_backward(r, x, w, dsum=r, stream=side))
    side.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ptc.rms_norm(x, w, residual=r), ptc.rms_norm_s8(x, w), ptc.rms_norm_backward(r, x, w, dsum=r)
    x0 = x.clone()
    x.copy_(rand(9, 300, 777, dtype=torch.bfloat16))
    graph.replay()
    x.copy_(x0)
    graph.replay()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_past_32_bit_offsets():
    """Rows whose offsets exceed 2^32 elements, by their pitch."""
    buf = torch.empty((1 << 32) + 4096, dtype=torch.bfloat16, device=DEV)
    v = buf.as_strided((3, 512), (1 << 31, 1))
    x = rand(1, 3, 512, dtype=torch.bfloat16)
    v.copy_(x)
    assert torch.equal(ptc.rms_norm(v), ptc.rms_norm(x))
    out = buf.as_strided((3, 512), (1 << 31, 1), 1024)
    assert torch.equal(ptc.rms_norm(x, out=out), ptc.rms_norm(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", [1, 7, 8, 9, 33, 250, 1000, 5003, 20001])
def test_s8_rows_at_any_element(cols, dtype):
    """Rows that begin at every element of a 16-byte word, with weights that do too: the codes are
    those of the same numbers in aligned rows, bit for bit (no code depends on a sum's order).
    The scale's 1 / rms may: either is within F32 of the formula's."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    rows = 5
    # (numbers around the ones that are read: none of them may count)
    wide = torch.full((rows, cols + 24), 1e4, device="cuda").to(dtype)
    wide_w = torch.full((cols + 24,), 1e3, device="cuda").to(dtype)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
    w = torch.randn(cols, generator=g, device="cuda").to(dtype)
    aligned = torch.zeros(rows, -(-cols // 8) * 8, device="cuda", dtype=dtype)[:, :cols]
    aligned.copy_(x)
    want, want_scale = ptc.rms_norm_s8(aligned, w)
    for off in range(9):
        part, part_w = wide[:, off:off + cols], wide_w[off:off + cols]
        part.copy_(x)
        part_w.copy_(w)
        got, scale = ptc.rms_norm_s8(part, part_w)
        assert torch.equal(got, want), off
        assert ((scale - want_scale).abs() <= 2 * F32 * want_scale.abs()).all(), off
        wide.fill_(1e4)
        wide_w.fill_(1e3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows", [5, 400])
@pytest.mark.parametrize("cols", [1, 7, 8, 9, 33, 250, 1001, 5003, 20001])
def test_rows_that_lie_alike(cols, rows, dtype):
    """Every matrix of a call begins at the same element of a 16-byte word, each of them in turn, in
    rows of any pitch: the formula's values, and nothing written beside them."""
    pitch = cols + 24
    x, r, w = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype), rand(3, cols, dtype=dtype)
    s = x + r
    v = s.double()
    want = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    for off in range(8) if rows == 5 else (0, 3):
        for weight in (w, torch.cat([w[:1], w])[1:]):
            wide = [torch.full((rows, pitch), 7.0, device=DEV).to(dtype) for _ in range(4)]
            px, pr, py, ps = (b[:, off:off + cols] for b in wide)
            px.copy_(x)
            pr.copy_(r)
            ptc.rms_norm(px, weight, 1e-6, residual=pr, out=py, sum_out=ps)
            assert torch.equal(ps, s) and torch.equal(px, x), off
            near(py, want, dtype)
            for b in wide[2:]:
                assert (b[:, :off] == 7).all() and (b[:, off + cols:] == 7).all(), off


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("cols", [1, 7, 9, 33, 250, 1001, 5003, 9001])
def test_gradient_of_rows_that_lie_alike(cols, rows, dtype):
    """The same for the gradient, whose rows of odd length begin at other elements one after the
    other: NaN beside the rows counts nowhere, and the values are those of separate rows."""
    s, dy, ds, w = (rand(k, *shape, dtype=dtype) for k, shape in enumerate([(rows, cols)] * 3 + [(cols,)]))
    pad = torch.full((rows, -(-cols // 8) * 8 + 8), float("nan"), device=DEV).to(dtype)

    def apart(t):  # 16-byte aligned rows
        b = pad.clone()
        b[:, :cols].copy_(t)
        return b[:, :cols]

    want, want_w = ptc.rms_norm_backward(apart(dy), apart(s), w, 1e-6, dsum=apart(ds), out=apart(dy))
    for off in range(8) if rows == 5 else (0, 3):
        for pitch in (cols + 8, cols + 9):
            wide = [torch.full((rows, pitch), float("nan"), device=DEV).to(dtype) for _ in range(4)]
            part = [b[:, off:off + cols] for b in wide]
            for to, t in zip(part, (s, dy, ds)):
                to.copy_(t)
            got, got_w = ptc.rms_norm_backward(part[1], part[0], w, 1e-6, dsum=part[2], out=part[3])
            assert got.data_ptr() == part[3].data_ptr()
            # Both are within the type's rounding and 2 F32 of terms no larger than these.
            v, g = s.double(), dy.double() * w.double()
            r = (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()
            size = r * (g.abs() + (v * r).abs() * (g * v * r).abs().mean(1, keepdim=True)) + ds.double().abs()
            bound = 2 * (ulp(dtype) * (want.double().abs() + 2 * F32 * size) + 2 * F32 * size + least(dtype))
            assert bool(((got.double() - want.double()).abs() <= bound).all()), off
            bound = 2 * (2 * F32 + (rows + 40) * 2.0 ** -24) * (dy.double() * v * r).abs().sum(0)
            assert bool(((got_w.double() - want_w.double()).abs() <= bound + 1e-30).all()), off
            assert bool(wide[3][:, :off].isnan().all()) and bool(wide[3][:, off + cols:].isnan().all())
