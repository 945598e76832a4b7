"""Workspaces on another GPU than the call's tensors are refused."""
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_gradient_reduction_amd as sg

if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)


def test_another_gpu():
    with FakeTensorMode():
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda:1")
        x, row, mean = torch.empty(6, 64, device="cuda:0"), torch.empty(64, device="cuda:0"), torch.empty(6, device="cuda:0")
        flat, heads, lse = torch.empty(4096, device="cuda:0"), torch.empty(1, 6, 2, 64, device="cuda:0"), torch.empty(1, 2, 6, device="cuda:0")
        for call in (lambda: sg.layer_norm_backward(x, x, row, mean, mean, workspace=ws),
                     lambda: sg.orthogonalize(flat, [(0, 64, 64)], workspace=ws),
                     lambda: sg.orthogonal_step(flat, flat, [(0, 64, 64)], lr=0.1, workspace=ws),
                     lambda: sg.head_norm_rotate_backward(heads, heads, heads, heads, workspace=ws),
                     lambda: sg.attention_backward(heads, heads, heads, heads, heads, lse, workspace=ws)):
            with pytest.raises(ValueError, match="workspace must be on cuda:0"):
                call()
