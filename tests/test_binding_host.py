"""What the Python binding takes as an address."""

import fractions

import numpy as np
import pytest
import torch

import group_quantized_mat_gb300 as g


def test_tensors_arrays_and_integers_are_addresses():
    t, n = torch.zeros(4), np.zeros(4)
    assert g._ptr(t) == t.data_ptr() and g._ptr(t[1:]) == t.data_ptr() + 4
    assert g._ptr(n) == n.ctypes.data and g._ptr(1 << 40) == 1 << 40 and g._ptr(0) == 0 and g._ptr(None) is None


@pytest.mark.parametrize("bad", [1.0, 4096.0, "4096", b"4096", [4096], (1,), fractions.Fraction(16), np.float32(16), np.int64(16), object()])
def test_nothing_else_is(bad):
    with pytest.raises(AttributeError):
        g._ptr(bad)


def test_a_call_refuses_what_is_no_address():
    from group_quantized_mat_gb300 import build
    build.build()
    fake = 1 << 20
    for bad in (float(fake), str(fake)):
        with pytest.raises(AttributeError):
            g.qmv_run(fake, fake, fake, bad, fake, 0, 64, 64, 4, 64, stream=0)
