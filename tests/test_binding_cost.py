"""The binding's argument conversion takes no detour through an exception for
what every entry point is called with: missing tensors, tensors, pointers, and
the shapes of the layer, the sorted rows and the 4-bit weights."""
import ctypes
import sys

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib

ARGS = {
    "none": (_lib._p, None), "tensor": (_lib._p, torch.zeros(3)), "pointer": (_lib._p, 4096),
    "layer": (_lib._shape, m.Shape(4, 64, 8, 2, 64)),
    "struct": (_lib._shape, m.Shape(4, 64, 8, 2, 64).c()),
    "rows": (_lib._shape, m.SortShape(4, 8, 2, 64)),
    "w4": (_lib._shape, m.W4Shape(1, 16, 32)),
    "experts": (_lib._shape, m.W4Experts(*[torch.zeros(1)] * 3)),
}


@pytest.mark.parametrize("name", list(ARGS))
def test_no_exception_on_the_way(name):
    fn, arg = ARGS[name]
    fn(arg)  # shapes make their struct at the first call
    raised = []

    def trace(frame, event, _):
        if event == "exception":
            raised.append(frame.f_code.co_name)
        return trace
    before = sys.gettrace()
    sys.settrace(trace)
    try:
        got = fn(arg)
    finally:
        sys.settrace(before)
    assert not raised
    if fn is _lib._p:
        assert got == (arg if arg is None or isinstance(arg, int) else arg.data_ptr())
    else:
        assert type(got) is type(ctypes.byref(ctypes.c_int()))


def test_what_is_no_argument_raises():
    with pytest.raises((AttributeError, TypeError)):
        _lib._p("x")
    with pytest.raises((AttributeError, TypeError)):
        _lib._shape(None)
