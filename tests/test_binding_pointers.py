"""How the binding takes addresses: tensors, whole numbers, host arrays, none."""
import sys

import numpy as np
import pytest
import torch

import weight_quantized_gemm_gb300 as qg


class Address(int):
    pass


@pytest.mark.parametrize("x", [1 << 40, 0, Address(1 << 41), True])
def test_whole_numbers(x):
    assert qg._ptr(x) == int(x)


def test_tensors_arrays_and_none():
    t, a = torch.zeros(4), np.zeros(4)
    assert qg._ptr(t) == t.data_ptr() and qg._ptr(a) == a.ctypes.data and qg._ptr(None) is None


def test_an_address_raises_nothing_on_its_way():
    """A call takes up to ten addresses; one raised and caught inside for each would take longer than the call."""
    raised = []

    def trace(frame, event, arg):
        if event == "exception":
            raised.append(arg[0])
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        qg._ptr(1 << 40)
        qg._ptr(None)
    finally:
        sys.settrace(before)
    assert not raised
