"""The binding's way from an argument to an address: tensors, arrays, plain addresses and None, the last three without the
cost of an exception."""

import enum
import sys

import numpy as np
import pytest


class Address(enum.IntEnum):
    A = 4096


def raised_in(code, f, x):
    """f(x), and the exceptions that were raised in `code` on the way."""
    seen = []

    def trace(frame, event, arg):
        if event == "exception" and frame.f_code is code:
            seen.append(arg[0])
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        return f(x), seen
    finally:
        sys.settrace(before)


def test_addresses(ekv_lib):
    torch = pytest.importorskip("torch")
    f, a, t = ekv_lib._ptr, np.zeros(4), torch.zeros(4)
    for x, want in ((None, None), (0, 0), (1 << 40, 1 << 40), (a, a.ctypes.data), (a[1:], a.ctypes.data + 8), (t, t.data_ptr()),
                    (t[2:], t.data_ptr() + 8)):
        assert raised_in(f.__code__, f, x) == (want, [])
    assert f(Address.A) == 4096 and f(a.view(np.recarray)) == a.ctypes.data
    for x in ("a", 1.5, object()):
        with pytest.raises(TypeError):
            f(x)
