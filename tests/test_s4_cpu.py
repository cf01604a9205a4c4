"""Refusals of the grouped 4-bit integer product before any CUDA call, and the weights'
layout, on the CPU."""
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


def product(L, M=4, N=40, K=200, type=1, X=BASE, ldx=200, W=BASE + GB, ldw=112, group=64, st=1, scales=BASE + 2 * GB,
            zeros=None, C=BASE + 4 * GB, ldc=40, ws=None, bytes=0):
    return L.gemm_a16_s4(M, N, K, type, X, ldx, W, ldw, group, st, scales, zeros, C, ldc, ws, bytes, None)


@no_gpu
@pytest.mark.parametrize("change, status", [
    (dict(), DEVICE), (dict(M=-1), INVALID), (dict(K=(1 << 30) + 1), INVALID), (dict(M=65535 * 16 + 1), INVALID),
    (dict(M=0, X=None, C=None), 0), (dict(N=0), 0), (dict(type=0), INVALID), (dict(st=0), INVALID), (dict(st=2), DEVICE),
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(scales=None), INVALID), (dict(C=None), INVALID),
    (dict(ldx=199), INVALID), (dict(ldw=96), INVALID), (dict(ldw=104), ALIGN), (dict(ldc=39), INVALID),
    (dict(group=0), INVALID), (dict(group=96), INVALID), (dict(group=16), INVALID), (dict(group=-128), INVALID),
    (dict(group=256), DEVICE), (dict(group=1 << 30), DEVICE), (dict(X=BASE + 1), ALIGN), (dict(W=BASE + GB + 8), ALIGN),
    (dict(scales=BASE + 2 * GB + 2), ALIGN), (dict(zeros=BASE + 3 * GB + 8), ALIGN), (dict(zeros=BASE + 3 * GB), DEVICE),
    (dict(C=BASE), OVERLAP), (dict(C=BASE + GB + 64), OVERLAP), (dict(C=BASE + 2 * GB + 3 * 4 * 32 - 2), OVERLAP),
    (dict(C=BASE + 2 * GB + 3 * 4 * 32), DEVICE), (dict(C=BASE + 3 * GB, zeros=BASE + 3 * GB), OVERLAP),
    (dict(K=0, X=None, W=None, scales=None), DEVICE), (dict(C=BASE + 400, ldx=240, ldc=240), DEVICE),
    (dict(ws=BASE + 5 * GB, bytes=4 * 512 + 8 * 64), DEVICE), (dict(ws=BASE + 5 * GB, bytes=4 * 512 + 8 * 64 - 1), INVALID),
    (dict(ws=BASE + 5 * GB + 8, bytes=1 << 20), ALIGN), (dict(ws=BASE, bytes=1 << 20), OVERLAP), (dict(ws=BASE + 4 * GB, bytes=1 << 20), OVERLAP),
    (dict(M=2, ws=BASE + 8, bytes=0), DEVICE),  # (not used)
])
def test_statuses(L, change, status):
    assert product(L, **change) == status


def test_tile_scales():
    """[tile][group][row of 16], experts in order, rows past the last filled up."""
    s = torch.arange(2 * 20 * 3).view(2, 20, 3).half()
    t = ptc.S4Matrix.tile_scales(s)
    assert t.numel() == 2 * 2 * 3 * 16
    for e in range(2):
        for r in range(20):
            for g in range(3):
                assert t[((e * 2 + r // 16) * 3 + g) * 16 + r % 16] == s[e, r, g]
    assert ptc.S4Matrix.tile_scales(torch.empty(0, 3)).numel() == 0


def test_host_tensors_are_refused():
    codes, scales = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ptc.S4Matrix(codes, scales, 32, 32)
    with pytest.raises(TypeError):
        ptc.S4Matrix(codes.int(), scales, 32, 32)
    with pytest.raises(TypeError):
        ptc.matmul_a16_s4(torch.zeros(1, 32), codes)


def test_keys(L):
    assert [L.ptc_set_tuning(b"s4_tokens_rows", v) for v in (16, 0)] == [0, 0] and L.ptc_set_tuning(b"s4_tokens_split", 16) == INVALID
    for key in (b"s4_tokens_rows", b"s4_tokens_split"):
        assert [L.ptc_set_tuning(key, v) for v in (1, 2, 4, 8, 0)] == [0] * 5
        assert L.ptc_set_tuning(key, 3) == INVALID and L.ptc_set_tuning(key, -1) == INVALID
    assert [L.ptc_set_tuning(b"s4_tokens_tiles", v) for v in (1, 2, 0, 3)] == [0, 0, 0, INVALID]


def moe(L, tokens=4, hidden=200, inner=100, experts=5, top_k=2, type=1, X=BASE, ldx=200, router=BASE + GB, ldr=200, rt=1, group=64,
        st=1, gu=BASE + 2 * GB, ldg=112, eg=200 * 112, gs=BASE + 3 * GB, gz=None, dn=BASE + 4 * GB, ldd=64, ed=200 * 64,
        ds=BASE + 5 * GB, dz=None, Y=BASE + 6 * GB, ldy=200, ids=None, weights=None, ws=BASE + 7 * GB, bytes=None):
    if bytes is None:
        bytes = L.ptc_moe_a16_s4_workspace(tokens, hidden, inner, experts, top_k)
    return L.ptc_moe_a16_s4(tokens, hidden, inner, experts, top_k, 1, type, X, ldx, router, ldr, rt, group, st, gu, ldg, eg, gs, gz,
                            dn, ldd, ed, ds, dz, Y, ldy, ids, weights, ws, bytes, None)


@no_gpu
@pytest.mark.parametrize("change, status", [
    (dict(), DEVICE), (dict(tokens=0, X=None), 0), (dict(tokens=65), INVALID), (dict(tokens=-1), INVALID), (dict(hidden=0), INVALID),
    (dict(inner=0), INVALID), (dict(experts=513), INVALID), (dict(top_k=0), INVALID), (dict(top_k=6), INVALID),
    (dict(experts=64, top_k=33), INVALID), (dict(tokens=64, experts=64, top_k=9), INVALID), (dict(tokens=64, experts=64, top_k=8), DEVICE),
    (dict(type=0), INVALID), (dict(rt=2), INVALID), (dict(rt=0), DEVICE), (dict(st=0), INVALID), (dict(st=2), DEVICE),
    (dict(group=48), INVALID), (dict(ldx=199), INVALID), (dict(ldy=199), INVALID), (dict(ldr=199), INVALID), (dict(ldg=96), INVALID),
    (dict(ldd=48), INVALID), (dict(eg=200 * 112 - 16), INVALID), (dict(ed=16), INVALID), (dict(ed=200 * 64 + 8), ALIGN),
    (dict(gu=None), INVALID), (dict(ds=None), INVALID), (dict(gu=BASE + 2 * GB + 8), ALIGN), (dict(dz=BASE + 8 * GB + 2), ALIGN),
    (dict(X=BASE + 1), ALIGN), (dict(ids=BASE + 8 * GB + 2), ALIGN), (dict(ids=BASE + 8 * GB, weights=BASE + 9 * GB), DEVICE),
    (dict(ws=None), INVALID), (dict(ws=BASE + 7 * GB + 128), ALIGN), (dict(bytes=1000), INVALID), (dict(Y=BASE), OVERLAP),
    (dict(Y=BASE + 4 * GB + 64), OVERLAP), (dict(weights=BASE + 7 * GB), OVERLAP), (dict(ids=BASE + 8 * GB, weights=BASE + 8 * GB), OVERLAP),
    (dict(Y=BASE + 2 * GB + 5 * 200 * 112 - 16), OVERLAP), (dict(ws=BASE + 5 * GB), OVERLAP),
])
def test_moe_statuses(L, change, status):
    assert moe(L, **change) == status


def test_moe_workspace():
    f = ptc.ptc_moe_a16_s4_workspace
    assert f(0, 1, 1, 1, 1) == f(65, 1, 1, 1, 1) == f(1, 0, 1, 1, 1) == f(1, 1, 1, 1, 2) == f(64, 1, 1, 64, 9) == 0
    # counters, logits, operands of x and their factors, of h and theirs, shares of y
    assert f(3, 300, 200, 10, 2) == 4352 + 256 + 3 * 2 * 512 + 512 + 6 * 1024 + 512 + 2048 * 3 * 64
