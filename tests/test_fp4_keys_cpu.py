"""The few-token product's keys and the record of the last 4-bit launch, without a GPU."""
import ctypes

import pytest

import precision_tensor_core_gb300 as ptc


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_tuning_keys():
    for key in ("fp4_tokens_rows", "fp4_tokens_split"):
        for bad in (-1, 3, 16):
            with pytest.raises(ptc.PtcError):
                ptc.ptc_set_tuning(key, bad)
        for good in (1, 2, 4, 8, 0):
            assert ptc.ptc_set_tuning(key, good) == 0


def test_last_launch():
    assert len(ptc.ptc_last_fp4_launch()) == 4
    n = ctypes.c_int64(0)
    assert ptc.lib().ptc_last_fp4_launch(ctypes.byref(n), None, None, None) == ptc.PTC_ERR_INVALID
