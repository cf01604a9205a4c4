"""Refusals of the norms, before any CUDA call: statuses of the C entry points with
addresses that are never dereferenced, and the tensor layer's checks."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc

BASE, GB = 1 << 40, 1 << 30
INVALID, ALIGN, OVERLAP, DEVICE = ptc.PTC_ERR_INVALID, ptc.PTC_ERR_ALIGN, ptc.PTC_ERR_OVERLAP, ptc.PTC_ERR_DEVICE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would run")


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return ptc.lib()


def norm(L, rows=4, cols=24, x=BASE, ldx=24, type=1, res=None, ldr=0, sum=None, lds=0, w=None, wt=1, eps=1e-6,
         y=BASE + GB, ldy=24):
    return L.ptc_rms_norm(rows, cols, x, ldx, type, res, ldr, sum, lds, w, wt, eps, y, ldy, None)


def norm_s8(L, rows=4, cols=24, x=BASE, ldx=24, type=1, w=None, wt=1, eps=1e-6, y=BASE + GB, ldy=24, scale=BASE + 2 * GB):
    return L.ptc_rms_norm_s8(rows, cols, x, ldx, type, None, 0, None, 0, w, wt, eps, y, ldy, scale, None)


def grad(L, rows=4, cols=24, dy=BASE, s=BASE + GB, type=1, ds=None, w=None, wt=1, eps=1e-6, dx=BASE + 2 * GB, ld=24,
         dw=BASE + 3 * GB, ws=BASE + 4 * GB, bytes=None):
    need = L.ptc_rms_norm_backward_workspace(rows, cols) if bytes is None else bytes
    return L.ptc_rms_norm_backward(rows, cols, dy, ld, s, ld, type, ds, ld, w, wt, eps, dx, ld, dw, ws, need, None)


@no_gpu
@pytest.mark.parametrize("change, status", [
    (dict(), DEVICE), (dict(rows=-1), INVALID), (dict(cols=(1 << 30) + 1), INVALID), (dict(rows=0, x=None, y=None), 0),
    (dict(cols=0), 0), (dict(type=3), INVALID), (dict(wt=2), INVALID), (dict(wt=0), DEVICE), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(ldx=23), INVALID), (dict(ldy=(1 << 36) + 1), INVALID), (dict(x=BASE + 1), ALIGN), (dict(y=BASE + GB + 1), ALIGN),
    (dict(w=BASE + 2 * GB + 1), ALIGN), (dict(y=BASE), DEVICE), (dict(y=BASE + 2), OVERLAP), (dict(y=BASE, ldy=25), OVERLAP),
    (dict(y=BASE + 48, ldx=48, ldy=48), DEVICE),  # the other half of one buffer's rows
    (dict(sum=BASE + 2 * GB, lds=24), INVALID), (dict(res=BASE + 2 * GB, ldr=24), INVALID),
    (dict(res=BASE + 2 * GB, ldr=24, sum=BASE + 3 * GB, lds=24), DEVICE),
    (dict(res=BASE + 2 * GB, ldr=24, sum=BASE + 2 * GB, lds=24), DEVICE),  # the residual stream in place
    (dict(res=BASE + 2 * GB, ldr=24, sum=BASE + 2 * GB, lds=24, y=BASE), DEVICE),
    (dict(res=BASE + 2 * GB, ldr=24, sum=BASE + GB, lds=24), OVERLAP),  # sum and y
    (dict(res=BASE + 2 * GB, ldr=24, sum=BASE + 2 * GB + 2, lds=24), OVERLAP), (dict(w=BASE + GB), OVERLAP),
])
def test_norm_statuses(L, change, status):
    assert norm(L, **change) == status


@no_gpu
@pytest.mark.parametrize("change, status", [
    (dict(), DEVICE), (dict(scale=None), INVALID), (dict(scale=BASE + 2 * GB + 2), ALIGN), (dict(y=BASE), OVERLAP),
    (dict(y=None), INVALID), (dict(scale=BASE + GB + 8), OVERLAP), (dict(scale=BASE + 4), OVERLAP), (dict(ldy=23), INVALID),
    (dict(y=BASE + GB + 1), DEVICE),  # bytes have no alignment
])
def test_norm_s8_statuses(L, change, status):
    assert norm_s8(L, **change) == status


@no_gpu
@pytest.mark.parametrize("change, status", [
    (dict(), DEVICE), (dict(dw=None), INVALID), (dict(dw=BASE + 3 * GB + 2), ALIGN), (dict(ws=None), INVALID),
    (dict(bytes=4 * 24 * 4 - 1), INVALID), (dict(bytes=4 * 24 * 4), DEVICE), (dict(ws=BASE + 4 * GB + 8), ALIGN),
    (dict(dx=BASE), DEVICE), (dict(dx=BASE + GB), DEVICE), (dict(dx=BASE + 2), OVERLAP), (dict(dw=BASE + 4 * GB), OVERLAP),
    (dict(dw=BASE), OVERLAP), (dict(ws=BASE + GB), OVERLAP), (dict(cols=0), 0), (dict(s=None), INVALID), (dict(ld=20), INVALID),
    (dict(ds=BASE + 5 * GB, dx=BASE + 5 * GB), DEVICE), (dict(rows=0), DEVICE), (dict(eps=-0.5), INVALID),
])
def test_norm_backward_statuses(L, change, status):
    assert grad(L, **change) == status


def test_workspace_sizes(L):
    f = ptc.ptc_rms_norm_backward_workspace
    assert f(0, 10) == f(10, 0) == f(-1, 5) == 0
    assert f(3, 100) == 3 * 100 * 4 and f(10 ** 6, 100) == 512 * 100 * 4
    assert f(3, 20000) >= 3 * 20000 * 4 + 3 * 8


def test_host_tensors_and_wrong_arguments_are_refused():
    x = torch.zeros(3, 8)
    for call in (lambda: ptc.rms_norm(x), lambda: ptc.rms_norm_s8(x), lambda: ptc.rms_norm_backward(x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        ptc.rms_norm(x.int())
    with pytest.raises(TypeError):
        ptc.rms_norm([1.0])
    with pytest.raises(RuntimeError, match="requires grad"):
        ptc.rms_norm(x.requires_grad_())
