"""Which arguments share bytes: rows that lie side by side in one buffer do not.

Without a GPU a call that is not refused stops at the device check, so these
only run where there is none (the addresses are never dereferenced)."""
import pytest
import torch

import precision_tensor_core_gb300 as ptc

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would run")
BASE, GB = 1 << 40, 1 << 30


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return ptc.lib()


def dropout(L, rows, cols, x, ldx, y, ldy, r=None, ldr=0):
    return L.ptc_dropout(rows, cols, x, ldx, r, ldr, y, ldy, 1, 0.5, 1, 0, None)


@pytest.mark.parametrize("rows", [1, 2, 40])
def test_every_offset_against_the_bytes_themselves(L, rows):
    """x at element 100, y everywhere around it, compared with the sets of elements (equal pitches)."""
    for ld, cols in ((12, 5), (12, 6), (12, 7), (7, 7)):
        xs = {100 + i * ld + j for i in range(rows) for j in range(cols)}
        for at in range(100 - 3 * ld, 100 + (rows + 2) * ld):
            if at == 100:
                continue
            ys = {at + i * ld + j for i in range(rows) for j in range(cols)}
            spans_meet = not (max(ys) < min(xs) or max(xs) < min(ys))
            got = dropout(L, rows, cols, BASE + 200, ld, BASE + 2 * at, ld)
            if xs & ys:
                assert got == ptc.PTC_ERR_OVERLAP, (ld, cols, at)
            elif spans_meet and (at - 100) % ld >= cols and (at - 100) % ld + cols <= ld:
                assert got == ptc.PTC_ERR_DEVICE, (ld, cols, at)  # between x's columns
            elif not spans_meet:
                assert got == ptc.PTC_ERR_DEVICE, (ld, cols, at)


def test_other_pitches_and_other_operators(L):
    assert dropout(L, 10, 40, BASE, 100, BASE + 80, 200) == ptc.PTC_ERR_OVERLAP
    assert dropout(L, 10, 40, BASE, 100, BASE + 80, 100, r=BASE + 120, ldr=100) == ptc.PTC_ERR_OVERLAP
    assert dropout(L, 10, 30, BASE, 100, BASE + 80, 100, r=BASE + 140, ldr=100) == ptc.PTC_ERR_DEVICE

    def tokens(C, ldc):
        return L.gemm_a16_fp4(7, 96, 160, 1, BASE, 264, 0, BASE + GB, 80, BASE + 2 * GB, None, C, ldc, None)

    assert tokens(BASE + 2 * 160, 264) == ptc.PTC_ERR_DEVICE
    for C, ldc in ((BASE + 2 * 159, 264), (BASE + 2 * 169, 264), (BASE + 2 * 160, 272), (BASE + GB + 80 * 95, 264)):
        assert tokens(C, ldc) == ptc.PTC_ERR_OVERLAP

    def product(A, lda, C, ldc):  # codes of A beside the 16-bit results in one buffer
        return L.gemm_fp4(20, 64, 64, 0, A, lda, BASE + GB, None, BASE + 2 * GB, 32, BASE + 3 * GB, None, C, ldc, 1, None)

    assert product(BASE, 256, BASE + 32, 128) == ptc.PTC_ERR_DEVICE
    assert product(BASE + 128, 256, BASE, 128) == ptc.PTC_ERR_DEVICE
    assert product(BASE + 112, 256, BASE, 128) == ptc.PTC_ERR_OVERLAP
