"""Addresses as the binding takes them: a number is one at once (asked for
data_ptr() first, each cost a raised exception, 1.2 us)."""
import numpy as np
import pytest

import matmul_selection_gb300 as mm


class Address(int):
    def data_ptr(self):
        raise RuntimeError("a number was asked for its address")


class Tensor:
    def data_ptr(self):
        return 0x1000


def test_numbers_tensors_arrays():
    assert mm._ptr(Address(0x2000)) == 0x2000
    assert mm._ptr(None) is None
    assert mm._ptr(Tensor()) == 0x1000
    a = np.zeros(4)
    assert mm._ptr(a) == a.ctypes.data
    with pytest.raises(TypeError):
        mm._ptr("x")


@pytest.mark.parametrize("fast", [mm._fast, mm._Ctypes])
@pytest.mark.parametrize("t", [1 << 32, -(1 << 32), (1 << 32) + 1, 1 << 31])
def test_types_past_32_bits_are_no_types(t, fast, monkeypatch):
    monkeypatch.setattr(mm, "_fast", fast)
    for dt in ((t, 0, 0), (0, t, 0), (0, 0, t)):
        assert mm.mm_rmsnorm(2, None, 2, None, 4, None, None, 1, 1, 1, 1, 1, 1, dt, 0.0) == mm.MM_ERR_INVALID_ARG
        assert "types" in mm.mm_last_error()
