"""What ptc_dropout_to refuses, before any CUDA call (the addresses are never dereferenced)."""
import pytest

import precision_tensor_core_gb300 as ptc

BASE, GB = 1 << 40, 1 << 30


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return ptc.lib()


def test_refusals(L):
    def call(rows=4, cols=100, x=BASE, ldx=100, type=0, r=None, ldr=0, y=BASE + GB, ldy=100, out=1, p=0.5, offset=0):
        return L.ptc_dropout_to(rows, cols, x, ldx, type, r, ldr, y, ldy, out, p, 1, offset, None)

    for bad in (dict(type=1, out=0), dict(type=1, out=2), dict(out=3), dict(type=-1), dict(r=BASE + 2 * GB, ldr=100),
                dict(x=None), dict(y=None), dict(ldx=99), dict(ldy=99), dict(p=2.0), dict(offset=1 << 63)):
        assert call(**bad) == ptc.PTC_ERR_INVALID, bad
    for bad in (dict(x=BASE + 2), dict(y=BASE + GB + 1)):
        assert call(**bad) == ptc.PTC_ERR_ALIGN, bad
    for bad in (dict(y=BASE), dict(y=BASE + 400 * 4 - 2), dict(type=0, out=0, y=BASE + 4)):
        assert call(**bad) == ptc.PTC_ERR_OVERLAP, bad
    assert call(cols=0, x=None, y=None) == ptc.PTC_OK
