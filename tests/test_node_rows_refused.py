"""Gradients of weights that lie on another GPU than the call's tensors are refused."""
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_gradient_reduction_amd as sg

if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)


def test_another_gpu():
    with FakeTensorMode():
        q, other = torch.empty(6, 4, 64, device="cuda:0"), torch.empty(1, 64, device="cuda:1")
        near = torch.empty(1, 64, device="cuda:0")
        for given in ({"dq_weight": other}, {"dk_weight": other}, {"dq_weight": near, "dk_weight": other}):
            with pytest.raises(ValueError):
                sg.head_norm_rotate_backward(q, q, q, q, **given)
        x, row, mean = torch.empty(6, 64, device="cuda:0"), torch.empty(64, device="cuda:0"), torch.empty(6, device="cuda:0")
        for given in ({"dweight": other}, {"dbias": other}):
            with pytest.raises(ValueError):
                sg.layer_norm_backward(x, x, row, mean, mean, **given)
