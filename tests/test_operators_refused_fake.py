"""What the dense operators' Python calls refuse of tensors on a GPU, on the
host: tensors without storage stand for the GPU's."""
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_gradient_reduction_amd as sg

if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)


@pytest.fixture
def fake():
    with FakeTensorMode():
        yield lambda *shape, t=torch.float32, device="cuda:0": torch.empty(shape, dtype=t, device=device)


@pytest.mark.parametrize("wrong", ["host", "fp32", "gaps"])
def test_workspaces(fake, wrong):
    """A workspace that is not bytes on a GPU never reaches a kernel."""
    ws = {"host": lambda: fake(1 << 20, t=torch.uint8, device="cpu"), "fp32": lambda: fake(1 << 20),
          "gaps": lambda: fake(1 << 20, 2, t=torch.uint8)[:, 0]}[wrong]()
    x, v, r = fake(4, 8), fake(8), fake(4)
    for call in (lambda: sg.layer_norm_backward(x, x, v, r, r, workspace=ws),
                 lambda: sg.orthogonalize(v, [(0, 2, 4)], workspace=ws),
                 lambda: sg.orthogonal_step(v, v, [(0, 2, 4)], lr=0.1, workspace=ws)):
        with pytest.raises(TypeError, match="workspace"):
            call()
