"""The scales that attention refuses, on the host."""
import ctypes
import math
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_gradient_reduction_amd as sg

if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)

from tests.test_attention_refused import A, Heads, attention_args


@pytest.mark.parametrize("scale", [1.01e30, 2.3e38, 3.4e38, 0.99e-30])
def test_the_calls(scale):
    """Past 2.36e38 the scale in base 2 would be infinite and every result NaN."""
    L, a = sg.lib(), attention_args(scale=scale)
    assert L.sparcml_attention(ctypes.addressof(a), A, 1 << 40, None) == sg.ERR_INVALID_ARG
    assert L.sparcml_attention_backward(ctypes.addressof(a), A, 1 << 40, None) == sg.ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_the_ends_are_taken(scale):
    none = Heads(0, 0, 0, 0)
    L, a = sg.lib(), attention_args(scale=scale, batch=0, q=none, k=none, v=none, out=none, lse=0, dout=none, dq=none, dk=none, dv=none)
    assert L.sparcml_attention(ctypes.addressof(a), None, 0, None) == sg.OK
    assert L.sparcml_attention_backward(ctypes.addressof(a), None, 0, None) == sg.OK


@pytest.mark.parametrize("scale", [1.01e30, 3e38, 1e39, 1e300, math.inf, math.nan, -1.0, 0.0, 0.99e-30])
def test_the_binding(scale):
    with FakeTensorMode():
        q, lse = torch.empty(2, 5, 4, 64, device="cuda:0"), torch.empty(2, 4, 5, device="cuda:0")
        with pytest.raises(ValueError):
            sg.attention(q, q, q, scale=scale)
        with pytest.raises(ValueError):
            sg.attention_backward(q, q, q, q, q, lse, scale=scale)
